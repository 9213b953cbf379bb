// Block-scaled 8-bit product for many token rows: a CTA pair (cta_group::2) owns 256 tokens x 256
// weight rows (SWIGLU: 128 gate and the 128 up rows of the same columns of h).
//
// out[t, n] = sum_b xs[t, b] ws[n / 128, b] (sum_{k in b} x[t, k] w[n, k]).  The tensor cores sum one
// k-block of 128 into one of two TMEM buffers (256 columns each); the eight promotion warps of
// each CTA add it, times one factor per row and weight block, to fp32 sums in registers: 128
// columns of one token per thread.  Tensor cores and promotion work on alternate buffers.  The
// pair halves what each SM reads: 32 KB per k-block of 512 MMA cycles.
//
// Warp 0 loads (TMA), warp 1 of the leading CTA issues MMAs, warps 4-11 promote and store; the
// first warpgroup hands registers to them.  A tile's sums are written while the MMAs of the next one's first two k-blocks run.
//
// Bound by the hand-over of the two buffers and, with few k-blocks to a tile, by the sums' way out.  A k-block takes 790 cycles
// (4096 x 4864 x 7168, four tiles to every pair): 512 of MMAs, and a buffer is the promotion's for about 1070 between two
// turns of them; tensor pipe 66% busy, issue slots 57%.  8192 x 12288 x 7168 471 us alone, 3.06 PFLOP/s (486 with the rows
// stored by the lanes), and 530 over seconds, when the power limit holds the clock at 1.66 of 2.07 GHz; fp32 492 and 555.
// Gate and up of 4096 tokens x 8 experts (7168 x 2048) 764 to 780 us, down 464 (508).
#include <atomic>
#include <type_traits>

#include "device.h"
#include "fp8_tc.cuh"
#include "launch.h"

namespace mse {
namespace routed {
namespace {

constexpr int kStages = 5;
constexpr int kPromoWarps = 8;
constexpr int kParts = kPromoWarps / 4;        // threads that share a token row
constexpr int kRun = 128 / kParts;             // columns in each of a thread's two runs
constexpr int kThreads = 128 + 32 * kPromoWarps;
// registers: 384 threads x 168 at launch = 128 x 56 + 256 x 224 afterwards
constexpr int kLaunchRegs = 168;
constexpr int kBand = 16;                       // token tiles whose weight tiles are taken in turn (L2 reuse)
constexpr uint32_t kStage = 2 * kOperandTile;  // per CTA: 128 token rows, 128 weight rows

struct PairCtrl {
    uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], drain;
    uint32_t tmem_base;
    int abort_flag;
    uint32_t amax[kParts][128];
};
constexpr uint32_t kStaged = 32 * 128;         // 32 rows of 128 bytes on their way out
constexpr uint32_t kStaging = 2 * kStaged;     // per promotion warp
constexpr size_t kSmem = kStages * (size_t)kStage + kPromoWarps * kStaging + 1024 + sizeof(PairCtrl) + 64;

// 32 lanes x 32 consecutive columns
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    return (uint32_t)f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16);
}

// shared -> global, 32 rows of 128 bytes, clipped to the tensor; its group is the issuing thread's
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *m, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// all but the newest N stores of this thread have read their shared memory
template <int N>
__device__ __forceinline__ void tma_store_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int EPI, int PARTS>
__global__ void __launch_bounds__(kThreads, 1)
    pair_block_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmOut, const BlockGemm g, const int n_tiles_n) {
    constexpr bool GLU = EPI == BLOCK_SWIGLU;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *staging = smem_raw + (base - raw) + kStages * kStage;
    PairCtrl *ctl = reinterpret_cast<PairCtrl *>(staging + kPromoWarps * kStaging);
    const int warp = __shfl_sync(~0u, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    // PARTS > 1: a cluster of PARTS pairs has one tile, each pair its share of the k-blocks
    const uint32_t in_cluster = cluster_ctarank(), rank = in_cluster & 1u, first_rank = in_cluster & ~1u;
    const int part = (int)(in_cluster >> 1);
    const bool leader = rank == 0;
    const int64_t cluster = blockIdx.x / (2 * PARTS), n_clusters = gridDim.x / (2 * PARTS);
    const int kb0 = (int)((int64_t)g.kb * part / PARTS), kb1 = (int)((int64_t)g.kb * (part + 1) / PARTS);
    const uint16_t both = (uint16_t)(0x3u << first_rank);
    volatile int *abort_flag = &ctl->abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&ctl->tfull[b]), 1);
            mbar_init(smem_u32(&ctl->tempty[b]), 2 * kPromoWarps);   // of both CTAs, on the leader's
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&ctl->tmem_base), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the peer's barriers are initialised before any remote use
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(~0u, ctl->tmem_base, 0);
    pdl_wait();
    if (g.tiles) pdl_launch_dependents();

    const int64_t slots = g.tiles ? *g.n_tiles : (g.T + 255) / 256;
    const int64_t total = slots * n_tiles_n;
    // tile id -> token tile z and weight tile n: bands of kBand token tiles, z fastest
    auto place = [&](int64_t id, Tile &t, int &n) {
        const int64_t per = (int64_t)kBand * n_tiles_n, band = id / per, in = id % per;
        const int64_t wide = min((int64_t)kBand, slots - band * kBand);
        (void)tile_of_slot(g, (int)(band * kBand + in % wide), t);
        n = (int)(in / wide);
    };

    int64_t issued = 0;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const bool el = elect_lane();
        if (warp == 0) {
            bool ok = true;
            int stage = 0;
            uint32_t phase = 0;
            for (int64_t id = cluster; ok && id < total; id += n_clusters) {
                Tile t;
                int n;
                place(id, t, n);
                const int x_row = t.row0 + (int)rank * 128;
                const int w_row = (int)(t.expert * g.w_group_rows) +
                                  (GLU ? n * 128 + (int)(rank * g.up_rows) : n * 256 + (int)rank * 128);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = warp_wait(smem_u32(&ctl->empty[stage]), phase ^ 1u, abort_flag, g);
                    if (!ok) break;
                    if (el) {
                        const uint32_t fb = map_to_rank(smem_u32(&ctl->full[stage]), first_rank), dst = base + stage * kStage;
                        if (leader) mbar_arrive_expect_tx(smem_u32(&ctl->full[stage]), 2 * kStage);
                        tma_load_2d_pair(dst, &tmX, fb, kb * kBlock, x_row);
                        tma_load_2d_pair(dst + kOperandTile, &tmW, fb, kb * kBlock, w_row);
                    }
                    __syncwarp();
                    ++issued;
                    if (++stage == kStages) { stage = 0; phase ^= 1u; }
                }
            }
        } else if (warp == 1 && leader) {
            const uint32_t idesc = idesc_e4m3_f32(256, 256);
            bool ok = true;
            int stage = 0;
            uint32_t phase = 0, use = 0;   // use: k-blocks so far; buffer use & 1
            for (int64_t id = cluster; ok && id < total; id += n_clusters) {
                for (int kb = kb0; kb < kb1; ++kb, ++use) {
                    const uint32_t b = use & 1u;
                    ok = warp_wait(smem_u32(&ctl->full[stage]), phase, abort_flag, g) &&
                         warp_wait(smem_u32(&ctl->tempty[b]), ((use >> 1) & 1u) ^ 1u, abort_flag, g);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t xd = smem_desc_sw128(base + stage * kStage);
                    const uint64_t wd = smem_desc_sw128(base + stage * kStage + kOperandTile);
                    if (el) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_e4m3_pair(tmem_base + b * 256u, xd + (uint64_t)(kk * 2), wd + (uint64_t)(kk * 2), idesc,
                                             kk > 0 ? 1u : 0u);
                        tc_commit_pair_multicast(smem_u32(&ctl->tfull[b]), both);
                        tc_commit_pair_multicast(smem_u32(&ctl->empty[stage]), both);
                    }
                    __syncwarp();
                    if (++stage == kStages) { stage = 0; phase ^= 1u; }
                }
            }
        }
        if constexpr (PARTS > 1) {   // the promotion warps' exchange
            __syncwarp();
            cluster_sync();
            cluster_sync();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int q = warp & 3, row = q * 32 + lane, share = (warp - 4) / 4;
        // this thread's columns: two runs (SWIGLU: of gate and of up)
        const uint32_t at0 = GLU ? share * kRun : share * 2 * kRun, at1 = GLU ? 128 + share * kRun : share * 2 * kRun + kRun;
        const uint32_t lanes = tmem_base + ((uint32_t)(q * 32) << 16);
        const uint32_t empty0 = map_to_rank(smem_u32(&ctl->tempty[0]), first_rank);
        const uint32_t empty1 = map_to_rank(smem_u32(&ctl->tempty[1]), first_rank);
        uint32_t use = 0, turn = 0;   // turn: of the two staging buffers
        // the next tile: its place and its first factors are on their way while this one's sums are written
        struct {
            Tile t;
            int n;
            const float *xs, *ws;
            float xa, ga, ua;
        } next;
        auto open = [&](int64_t id) {
            if (id >= total) return;
            place(id, next.t, next.n);
            const bool have = row < next.t.rows - (int)rank * 128;
            // factors of one k-block: xs (any valid row where this one is not), ws of the two runs (not by the read-only path:
            // this grid began while the kernel before it wrote xs)
            next.xs = g.xs + ((int64_t)next.t.row0 + (have ? (int)rank * 128 + row : 0)) * g.kb;
            const int blk = GLU ? next.n : min(2 * next.n + share * 2 * kRun / 128, (int)((g.N + kBlock - 1) / kBlock) - 1);
            next.ws = g.ws + (int64_t)next.t.expert * g.ws_group + (int64_t)blk * g.kb;
            next.xa = next.xs[kb0];
            next.ga = next.ws[kb0];
            next.ua = GLU ? next.ws[g.up_scales + kb0] : 0.f;
        };
        open(cluster);
        for (int64_t id = cluster; id < total; id += n_clusters) {
            const Tile t = next.t;
            const int n = next.n;
            const bool row_ok = row < t.rows - (int)rank * 128;
            const int64_t r = t.row0 + (int)rank * 128 + row;
            const float *xs = next.xs, *ws = next.ws;
            float acc[2 * kRun];
#pragma unroll
            for (int i = 0; i < 2 * kRun; ++i) acc[i] = 0.f;
            // one k-block ahead: a row's factors of 8 k-blocks share one 32-byte sector
            float xa = next.xa, ga = next.ga, ua = next.ua;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb, ++use) {
                const float f0 = xa * ga, f1 = GLU ? xa * ua : f0;
                if (kb + 1 < kb1) {
                    xa = xs[kb + 1];
                    ga = ws[kb + 1];
                    if (GLU) ua = ws[g.up_scales + kb + 1];
                }
                const uint32_t b = use & 1u;
                ok = warp_wait(smem_u32(&ctl->tfull[b]), (use >> 1) & 1u, abort_flag, g);
                if (!ok) break;
                tc_fence_after();
                const uint32_t src = lanes + b * 256u;
                // 32 columns are on their way from TMEM while the 32 before them are added
                uint32_t d[2][32];
                tmem_ld32(src + at0, d[0]);
#pragma unroll
                for (int c = 0; c < 2 * kRun; c += 32) {
                    const int then = c + 32;
                    tmem_ld_wait();
                    if (then < 2 * kRun) {
                        tmem_ld32(src + (then < kRun ? at0 + then : at1 + then - kRun), d[then / 32 & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster_relaxed(b ? empty1 : empty0);
                    }
#pragma unroll
                    for (int v = 0; v < 32; ++v)
                        acc[c + v] = fmaf(__uint_as_float(d[c / 32 & 1][v]), c < kRun ? f0 : f1, acc[c + v]);
                }
            }
            open(id + n_clusters);
            ok = named_barrier_and(1, 32 * kPromoWarps, ok);
            constexpr int cols = 2 * kRun / PARTS;   // of a thread's columns, those it finishes
            if constexpr (PARTS > 1) {
                // every pair gets a slice of the columns from all: [part][share][group of four columns][row]
                float4 *red = reinterpret_cast<float4 *>(smem_raw + (base - raw));
                constexpr int groups = cols / 4;
                static_assert((size_t)PARTS * kParts * groups * 128 * 16 <= kStages * (size_t)kStage, "exchange");
                cluster_sync();   // every ring of the cluster is idle
                if (ok) {
#pragma unroll
                    for (int i = 0; i < 2 * kRun / 4; ++i)
                        st_cluster_f32x4(map_to_rank(smem_u32(red + ((part * kParts + share) * groups + i % groups) * 128 + row),
                                                     (uint32_t)(2 * (i / groups)) + rank),
                                         make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]));
                }
                cluster_sync();
#pragma unroll
                for (int i = 0; i < groups; ++i) {
                    float4 v = red[(share * groups + i) * 128 + row];
#pragma unroll
                    for (int o = 1; o < PARTS; ++o) {   // in the order of the parts
                        const float4 w = red[((o * kParts + share) * groups + i) * 128 + row];
                        v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
                    }
                    acc[4 * i] = v.x;
                    acc[4 * i + 1] = v.y;
                    acc[4 * i + 2] = v.z;
                    acc[4 * i + 3] = v.w;
                }
            }
            if (!ok) break;
            if constexpr (GLU) {
                const int64_t j0 = (int64_t)n * kBlock + share * kRun;
#pragma unroll
                for (int i = 0; i < kRun; ++i) acc[i] = glu(acc[i], acc[kRun + i]);
                if (j0 + kRun > g.N) {   // columns of another weight, or of none
#pragma unroll
                    for (int i = 0; i < kRun; ++i)
                        if (j0 + i >= g.N) acc[i] = 0.f;
                }
                float most[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < kRun; ++i) most[i & 1] = abs_max_nan(most[i & 1], acc[i]);
                const uint32_t am = abs_bits(abs_max_nan(most[0], most[1]));
                ctl->amax[share][row] = am;
                named_barrier_sync(1, 32 * kPromoWarps);
                const float a = floored_amax(max(am, ctl->amax[share ^ 1][row]));
                // (the barrier after the next tile's k-blocks keeps the next write of amax behind this read)
                if (row_ok) {
                    const float inv = __fdiv_rn(kE4m3Max, a);   // h is in 32 bits: no ties to keep
                    uint8_t *dst = g.hq + r * g.ldh + j0;
#pragma unroll
                    for (int c = 0; c < kRun; c += 16) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float *v = acc + c + 4 * i;
                            w[i] = e4m3x2(v[0] * inv, v[1] * inv) | (e4m3x2(v[2] * inv, v[3] * inv) << 16);
                        }
                        // rows have a pitch of 16 bytes: a run that starts inside a row may be written whole
                        if (j0 + c < g.N) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (share == 0) g.hs[r * g.hb + n] = block_scale(a);
                }
            } else {
                // 128 bytes of each of the warp's 32 rows at a time through shared memory, so that a store
                // covers whole lines of four rows instead of 16 bytes of 32 (16-byte words of a row in
                // an order of their own, row mod 8, against bank conflicts)
                using Out = typename std::conditional<EPI == BLOCK_F32, float, uint16_t>::type;
                constexpr int kWord = 16 / sizeof(Out), kPass = 8 * kWord;   // columns in 16 and in 128 bytes
                const int64_t c0 = (int64_t)n * 256 + share * 2 * kRun + part * cols;
                Out *out = static_cast<Out *>(g.out);
                const bool aligned = ((reinterpret_cast<uintptr_t>(out) | (uint64_t)g.ldo * sizeof(Out)) & 15u) == 0;
                uint8_t *mine = staging + (warp - 4) * kStaging;
                const int64_t first = t.row0 + (int)rank * 128 + q * 32;
                const int left = min(t.rows - (int)rank * 128 - q * 32, 32);   // valid rows of this warp
                auto stage = [&](int c, uint8_t *mine) {   // columns c .. c + kPass of the warp's rows
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float *v = acc + c + i * kWord;
                        uint4 w;
                        if constexpr (EPI == BLOCK_F32) {
                            w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                           __float_as_uint(v[3]));
                        } else {
                            w = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                                           bf16x2(v[6], v[7]));
                        }
                        *reinterpret_cast<uint4 *>(mine + lane * 128 + (i ^ (lane & 7)) * 16) = w;
                    }
                    __syncwarp();
                };
                if (cols % kPass == 0 && aligned && left == 32) {
                    // whole rows of a warp leave by TMA, clipped at N, one buffer while the other is filled
#pragma unroll
                    for (int c = 0; c < cols; c += kPass) {
                        if (c0 + c >= g.N) break;
                        uint8_t *buf = mine + (turn++ & 1u) * kStaged;
                        if (lane == 0) tma_store_wait_read<1>();
                        __syncwarp();
                        stage(c, buf);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0)
                            tma_store_2d(&tmOut, smem_u32(buf), (int)((c0 + c) * (int64_t)sizeof(Out)), (int)first);
                    }
                } else if (left > 0) {
                    if (lane == 0) tma_store_wait_read<0>();
                    __syncwarp();
                    if (cols % kPass == 0 && aligned) {
#pragma unroll
                        for (int c = 0; c < cols; c += kPass) {
                            if (c0 + c >= g.N) break;
                            stage(c, mine);
                            const int64_t col = c0 + c + (lane & 7) * kWord;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int rr = i * 4 + lane / 8;
                                const uint4 w =
                                    *reinterpret_cast<const uint4 *>(mine + rr * 128 + ((lane & 7) ^ (rr & 7)) * 16);
                                Out *dst = out + (first + rr) * g.ldo + col;
                                if (rr < left && col + kWord <= g.N) {
                                    *reinterpret_cast<uint4 *>(dst) = w;
                                } else if (rr < left) {   // the rows' last, incomplete word
                                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                    for (int e = 0; e < kWord; ++e)
                                        if (col + e < g.N) {
                                            if constexpr (EPI == BLOCK_F32)
                                                dst[e] = __uint_as_float(u[e]);
                                            else
                                                dst[e] = (uint16_t)(u[e / 2] >> (e % 2 * 16));
                                        }
                                }
                            }
                            __syncwarp();
                        }
                    } else {   // rows that start anywhere: neighbouring columns by neighbouring lanes
#pragma unroll
                        for (int c = 0; c < cols; c += kPass) {
                            if (c0 + c >= g.N) break;
                            stage(c, mine);
                            for (int rr = 0; rr < left; ++rr)
#pragma unroll
                                for (int j = lane; j < kPass; j += 32)
                                    if (c + j < cols && c0 + c + j < g.N)
                                        out[(first + rr) * g.ldo + c0 + c + j] = *reinterpret_cast<const Out *>(
                                            mine + rr * 128 + ((j / kWord) ^ (rr & 7)) * 16 + j % kWord * sizeof(Out));
                            __syncwarp();
                        }
                    }
                }
            }
        }
        if (!GLU && lane == 0) tma_store_wait_all();
        __syncwarp();
    }

    // ---- teardown: every issued stage is released by the leader's MMA commit once its bytes (of both
    // CTAs) have landed and been used; after an abort the waits are bounded
    if (warp == 0 && lane == 0) {
        for (int64_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
            if (!mbar_wait_drain(smem_u32(&ctl->empty[i % kStages]), (uint32_t)((i / kStages) & 1),
                                 drain_limit(g.wait_limit_ns)))
                __nanosleep(200000);
    }
    if (warp == 1 && lane == 0 && leader) {
        tc_commit_pair_multicast(smem_u32(&ctl->drain), (uint16_t)(0x1u << first_rank));
        (void)mbar_wait_drain(smem_u32(&ctl->drain), 0, drain_limit(g.wait_limit_ns));
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

// Opts the kernel into its shared memory once per device.
template <int EPI, int PARTS>
cudaError_t prepare() {
    static std::atomic<uint64_t> done;   // bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (done.load(std::memory_order_acquire) >> (dev & 63) & 1)) return e;
    // the hand-over of registers needs the ones it was written for
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, pair_block_kernel<EPI, PARTS>)) != cudaSuccess) return e;
    if (at.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(pair_block_kernel<EPI, PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e == cudaSuccess) done.fetch_or(1ull << (dev & 63), std::memory_order_acq_rel);
    return e;
}

template <int EPI, int PARTS>
cudaError_t run(const CUtensorMap &tx, const CUtensorMap &tw, const CUtensorMap &to, const BlockGemm &g, int clusters,
                int n_tiles_n, bool pdl, cudaStream_t s) {
    const cudaError_t e = prepare<EPI, PARTS>();
    if (e != cudaSuccess) return e;
    return launch_kernel(pair_block_kernel<EPI, PARTS>, dim3((unsigned)(2 * PARTS * clusters)), kThreads, kSmem, pdl,
                         2 * PARTS, s, tx, tw, to, g, n_tiles_n);
}

// Clusters of PARTS pairs that can be resident at once (0 on failure).
template <int PARTS>
int resident_clusters() {
    static std::atomic<int> cache[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if ((n = cache[dev & 63].load()) > 0) return n;
    if (prepare<BLOCK_BF16, PARTS>() != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * PARTS);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * PARTS;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, pair_block_kernel<BLOCK_BF16, PARTS>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    cache[dev & 63].store(n);
    return n;
}

template <int EPI>
cudaError_t run_parts(int parts, const CUtensorMap &tx, const CUtensorMap &tw, const CUtensorMap &to, const BlockGemm &g,
                      int clusters, int n_tiles_n, bool pdl, cudaStream_t s) {
    switch (parts) {
        case 4: return run<EPI, 4>(tx, tw, to, g, clusters, n_tiles_n, pdl, s);
        case 2: return run<EPI, 2>(tx, tw, to, g, clusters, n_tiles_n, pdl, s);
        default: return run<EPI, 1>(tx, tw, to, g, clusters, n_tiles_n, pdl, s);
    }
}

}  // namespace

// Pairs that share a tile's k-blocks, where all tiles' clusters can be resident at once and the k-blocks saved
// are worth the exchange, 4 us with two pairs and 6 with four (us with one pair and split: 1024 x 2112 x 7168, 36 tiles,
// 26.1, 19.5; 256 x 7168 x 6144, 28 tiles, 23.2, 18.6; 512 x 4000 x 1000, 32 tiles of 8 k-blocks, 9.2, 10.4).
int pair_parts(int64_t tiles, int kb) {
    if (kb >= 24 && tiles <= resident_clusters<4>()) return 4;
    if (kb >= 16 && tiles <= resident_clusters<2>()) return 2;
    return 1;
}

namespace {
int pair_columns(const BlockGemm &g) {   // tiles of weight rows
    const int width = g.epi == BLOCK_SWIGLU ? 128 : 256;
    return (int)((g.N + width - 1) / width);
}
}  // namespace

Split pair_split(const BlockGemm &g, int sm_count) {
    const int64_t tiles = (g.tiles ? g.max_tiles : (g.T + 255) / 256) * pair_columns(g);
    const int parts = g.tiles ? 1 : pair_parts(tiles, g.kb);
    return {2 * parts * std::min<int64_t>(parts > 1 ? tiles : sm_count / 2, tiles), parts};
}

mse_status launch_block_pair(const BlockGemm &g, int sm_count, bool pdl, cudaStream_t s) {
    CUtensorMap tw, tx;
    mse_status st = map_bytes(&tw, g.wq, g.groups * g.w_group_rows, g.K, g.ldw, 128);
    if (st != MSE_OK) return st;
    if ((st = map_bytes(&tx, g.xq, g.T, g.K, g.ldx, 128)) != MSE_OK) return st;
    CUtensorMap to = tx;   // of rows at multiples of 16 bytes only
    const int64_t size = g.epi == BLOCK_F32 ? 4 : 2;
    if (g.epi != BLOCK_SWIGLU && ((reinterpret_cast<uintptr_t>(g.out) | (uint64_t)(g.ldo * size)) & 15u) == 0 &&
        (st = map_bytes(&to, g.out, g.T, g.N * size, g.ldo * size, 32)) != MSE_OK)
        return st;
    const int n_tiles_n = pair_columns(g);
    const Split split = pair_split(g, sm_count);
    const int parts = split.parts, clusters = (int)(split.ctas / (2 * parts));
    cudaError_t e;
    switch (g.epi) {
        case BLOCK_BF16: e = run_parts<BLOCK_BF16>(parts, tx, tw, to, g, clusters, n_tiles_n, pdl, s); break;
        case BLOCK_F32: e = run_parts<BLOCK_F32>(parts, tx, tw, to, g, clusters, n_tiles_n, pdl, s); break;
        default: e = run<BLOCK_SWIGLU, 1>(tx, tw, tx, g, clusters, n_tiles_n, pdl, s); break;
    }
    return e == cudaSuccess ? MSE_OK : MSE_ERR_CUDA;
}

}  // namespace routed
}  // namespace mse
