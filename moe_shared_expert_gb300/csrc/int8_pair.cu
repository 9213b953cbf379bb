// Product in 8-bit integers for many token rows: a CTA pair (cta_group::2) owns 256 weight rows x 256 tokens.
//
// Each CTA converts the 128 weight rows of its own (int8_tc.cuh) and loads half of the tokens, in fp16.  The sums have 256 TMEM
// columns, the converted weights the other 256 (four k-blocks).  A tile's tokens are two halves with barriers of their own: at the end
// of a chunk of k-blocks one half's sums are read while the MMAs of the other half run.
//
// Warp 0 loads (TMA), warp 1 of the leading CTA issues MMAs.  Warps 4-7 and 8-11 convert the weights of every other k-block each, and
// each has one half's sums: it reads them when a chunk ends, which is when it would next wait for room to convert into, and stores
// a tile some k-blocks later, while the MMAs have converted ones left.
//
// Bound by hand-overs and by the power limit.  A k-block brings 48 KB to each SM (tokens are two bytes here), which takes
// 0.48 to 0.56 us with the MMAs and the conversion left out (0.42 of it without the loads too: the way around four stages and
// slots, whose barriers lie in two SMs); its MMAs take 1024 cycles, 0.50 us at 2.07 GHz; together 0.68 to 0.75.  8192 x 12288 x 7168
// 815 us, 1.77 PFLOP/s, tensor pipe 71% busy at the 1.97 GHz that the power limit leaves; 8192 x 7168 x 2048 130 us.  Clusters of
// two pairs that share a tile's tokens by multicast take as long and find room for 72 of 76 pairs only.  With three stages and slots
// 10% more; more stages for the weights, set free by the converting warps, change nothing.
#include <atomic>

#include "device.h"
#include "int8_tc.cuh"
#include "launch.h"

namespace mse {
namespace sorted {
namespace {

constexpr int kStages = 4, kSlots = 4;               // k-blocks in shared memory, and of weights in TMEM
static_assert(kSlots <= kStages, "the order of waits before a conversion");
constexpr int kWorkWarps = 8, kThreads = 128 + 32 * kWorkWarps;
// registers: 384 threads x 168 at launch >= 128 x 56 + 256 x 224 afterwards
constexpr int kLaunchRegs = 168;
constexpr int kTokens = 256, kHalf = kTokens / 2;
constexpr int kBand = 8;                             // token tiles whose weight tiles are taken in turn (L2 reuse)
constexpr uint32_t kTokenBox = kHalf / 2 * 128;      // 64 tokens x 64 k, per CTA
constexpr uint32_t kTokenBytes = 4 * kTokenBox;
constexpr uint32_t kStage = kWeightTile + kTokenBytes;
constexpr int kMaxGroups = MSE_ROUTE_MAX_EXPERTS;

struct PairCtrl {
    uint64_t wfull[kStages], xfull[kStages], empty[kStages], afull[kSlots], aempty[kSlots], dfull[2], dempty[2], drain;
    uint32_t tmem_base;
    int abort_flag, slots;
    float xs[kWorkWarps][kHalf];
    int first[kMaxGroups], row0[kMaxGroups + 1];     // a group's first token tile, and its rows
    int end[kMaxGroups];
};
constexpr size_t kSmem = kStages * (size_t)kStage + 1024 + sizeof(PairCtrl) + 64;
static_assert(kSmem <= 227 * 1024, "shared memory");

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

// as mbar_wait_bounded, for a barrier on which both CTAs' threads arrive
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, volatile int *abort_flag, const Int8Gemm &g) {
    bool ok = mbar_try_wait_acq_cluster(bar, parity);
    if (!ok) {
        const uint64_t t0 = global_timer_ns();
        while (!(ok = mbar_try_wait_acq_cluster(bar, parity))) {
            if (*abort_flag) break;
            if (global_timer_ns() - t0 > g.wait_limit_ns) {
                *abort_flag = 1;
                raise_device_error(g.err, DEV_ERR_TIMEOUT);
                break;
            }
        }
    }
    return __all_sync(~0u, ok);
}

// PARTS 2: a cluster of two pairs has one tile, each pair half of its k-blocks and, at the end, half of its tokens.
template <int PARTS>
__global__ void __launch_bounds__(kThreads, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Int8Gemm g,
                     const int kb_total, const int n_tiles_n) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *ring = smem_raw + (base - raw);
    PairCtrl *ctl = reinterpret_cast<PairCtrl *>(ring + kStages * (size_t)kStage);
    const int warp = __shfl_sync(~0u, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const uint32_t in_cluster = cluster_ctarank(), rank = in_cluster & 1u, first_rank = in_cluster & ~1u;
    const bool leader = rank == 0;
    const uint16_t both = (uint16_t)(3u << first_rank);
    const int part = (int)(in_cluster >> 1);
    const int64_t pair = blockIdx.x / (2 * PARTS), n_pairs = gridDim.x / (2 * PARTS);   // (pairs that have tiles of their own)
    const int kb0 = kb_total * part / PARTS, kb = kb_total * (part + 1) / PARTS - kb0;
    volatile int *abort_flag = &ctl->abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&ctl->wfull[s]), 1);
            mbar_init(smem_u32(&ctl->xfull[s]), 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        for (int a = 0; a < kSlots; ++a) {
            mbar_init(smem_u32(&ctl->afull[a]), 8);     // four warps of both CTAs, on the leader's
            mbar_init(smem_u32(&ctl->aempty[a]), 1);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(smem_u32(&ctl->dfull[h]), 1);
            mbar_init(smem_u32(&ctl->dempty[h]), 8);    // four warps of either CTA, on the leader's
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&ctl->tmem_base), 512);
        tmem_relinquish_pair();
    }
    // The kernel before this one, of the same call, let this one start after its own wait: the offsets are complete.
    // (No more tiles than offsets that ascend can make, whatever they say: every number of a tile stays in 32 bits.)
    if (warp == 2) {
        const int most = (int)(g.T / kTokens + min((int64_t)g.groups, g.T));
        int before = 0;
        for (int g0 = 0; g.offsets && g0 < g.groups; g0 += 32) {
            const int i = g0 + lane;
            const int64_t a = i < g.groups ? min(max((int64_t)g.offsets[i], (int64_t)0), g.T) : 0;
            const int64_t b = i < g.groups ? min(max((int64_t)g.offsets[i + 1], (int64_t)0), g.T) : 0;
            const int tiles = b > a ? (int)((b - a + kTokens - 1) / kTokens) : 0;
            int upto = tiles;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(~0u, upto, d);
                if (lane >= d) upto += o;
            }
            if (i < g.groups) {
                ctl->first[i] = before + upto - tiles;
                ctl->row0[i] = (int)a;
                ctl->end[i] = (int)b;
            }
            before = min(before + __shfl_sync(~0u, upto, 31), most);
        }
        if (lane == 0) ctl->slots = g.offsets ? before : (int)((g.T + kTokens - 1) / kTokens);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the peer's barriers are initialised before any remote use
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(~0u, ctl->tmem_base, 0), tmem_a = tmem_base + kTokens;
    pdl_wait();

    // (PARTS 2: a cluster has one tile at most, whatever the offsets say)
    const int64_t slots = ctl->slots, total = PARTS > 1 ? min(slots * n_tiles_n, n_pairs) : slots * n_tiles_n;
    // tile id -> token tile and weight tile n: bands of kBand token tiles, the token tile fastest
    auto place = [&](int64_t id, RowTile &t, int &n) {
        const int64_t per = (int64_t)kBand * n_tiles_n, band = id / per, in = id % per;
        const int64_t wide = min((int64_t)kBand, slots - band * kBand);
        const int z = (int)(band * kBand + in % wide);
        n = (int)(in / wide);
        int lo = 0, skip = z;
        if (g.offsets) {
            for (int hi = g.groups; hi - lo > 1;) {   // the last group whose first tile is not behind z
                const int mid = (lo + hi) / 2;
                if (ctl->first[mid] <= z) lo = mid; else hi = mid;
            }
            skip = z - ctl->first[lo];
        }
        t.group = lo;
        t.row0 = (g.offsets ? ctl->row0[lo] : 0) + skip * kTokens;
        t.rows = (int)min((int64_t)kTokens, (g.offsets ? ctl->end[lo] : g.T) - t.row0);
    };

    int64_t issued = 0;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const bool el = elected();
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        if (warp == 0) {
            for (int64_t id = pair; ok && id < total; id += n_pairs) {
                RowTile t;
                int n;
                place(id, t, n);
                const int w_row = t.group * (int)g.N + n * 256 + (int)rank * 128;
                const int x_row = t.row0 + (int)rank * (kHalf / 2);
                for (int k = 0; k < kb; ++k) {
                    ok = wait_all(smem_u32(&ctl->empty[stage]), phase ^ 1u, abort_flag, g);
                    if (!ok) break;
                    if (el) {
                        const uint32_t dst = base + stage * kStage, wb = smem_u32(&ctl->wfull[stage]);
                        const uint32_t xb = map_to_rank(smem_u32(&ctl->xfull[stage]), first_rank);
                        mbar_arrive_expect_tx(wb, kWeightTile);
                        tma_load_2d_nohint(dst, &tmW, wb, (kb0 + k) * kInner, w_row);
                        const bool both = t.rows > kHalf;
                        if (leader) mbar_arrive_expect_tx(smem_u32(&ctl->xfull[stage]), both ? 2 * kTokenBytes : kTokenBytes);
#pragma unroll
                        for (int b = 0; b < 4; ++b)   // half b / 2, 64 k from b % 2; coordinates in bytes
                            if (b < 2 || both) tma_load_2d_pair(dst + kWeightTile + b * kTokenBox, &tmX, xb, (kb0 + k) * 2 * kInner + (b % 2) * 128,
                                             x_row + b / 2 * kHalf);
                    }
                    __syncwarp();
                    ++issued;
                    if (++stage == kStages) { stage = 0; phase ^= 1u; }
                }
            }
        } else if (warp == 1 && leader) {
            const uint32_t idesc = idesc_f16_f32(256, kHalf);
            uint32_t aphase = 0, use[2] = {0, 0};   // use: chunks of a half so far
            int a = 0;
            for (int64_t id = pair; ok && id < total; id += n_pairs) {
                RowTile t;
                int n;
                place(id, t, n);
                const int halves = t.rows > kHalf ? 2 : 1;
                for (int k = 0; k < kb; ++k) {
                    const int in = k % kChunkBlocks;
                    const bool last = in == kChunkBlocks - 1 || k == kb - 1;
                    ok = wait_all(smem_u32(&ctl->xfull[stage]), phase, abort_flag, g) &&
                         wait_cluster(smem_u32(&ctl->afull[a]), aphase, abort_flag, g);
                    if (!ok) break;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h == halves) break;
                        if (in == 0) {
                            ok = wait_cluster(smem_u32(&ctl->dempty[h]), (use[h] & 1u) ^ 1u, abort_flag, g);
                            if (!ok) break;
                        }
                        tc_fence_after();
                        const uint32_t x = base + stage * kStage + kWeightTile + h * 2 * kTokenBox;
                        if (el) {
#pragma unroll
                            for (int kk = 0; kk < kInner / 16; ++kk)
                                tc_mma_f16_ts_pair(tmem_base + h * kHalf, tmem_a + (uint32_t)(a * kATmem + kk * 8),
                                                   smem_desc_sw128(x + (kk / 4) * kTokenBox) + (uint64_t)(kk % 4 * 2), idesc,
                                                   in > 0 || kk > 0 ? 1u : 0u);
                            if (last) tc_commit_pair_multicast(smem_u32(&ctl->dfull[h]), both);
                        }
                        __syncwarp();
                        if (last) ++use[h];
                    }
                    if (!ok) break;
                    if (el) {
                        tc_commit_pair_multicast(smem_u32(&ctl->empty[stage]), both);
                        tc_commit_pair_multicast(smem_u32(&ctl->aempty[a]), both);
                    }
                    __syncwarp();
                    if (++stage == kStages) { stage = 0; phase ^= 1u; }
                    if (++a == kSlots) { a = 0; aphase ^= 1u; }
                }
            }
        }
        if constexpr (PARTS > 1) {   // the other warps' exchange
            __syncwarp();
            cluster_sync();
            cluster_sync();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int q = warp & 3, row = q * 32 + lane, h = (warp - 4) / 4;
        const uint32_t lanes = (uint32_t)(q * 32) << 16, src = tmem_base + (uint32_t)(h * kHalf) + lanes;
        const uint32_t dempty = map_to_rank(smem_u32(&ctl->dempty[h]), first_rank);
        float *xs = ctl->xs[warp - 4];
        const int chunks = (kb + kChunkBlocks - 1) / kChunkBlocks;
        const int64_t tiles = total > pair ? (total - pair + n_pairs - 1) / n_pairs : 0, blocks = tiles * kb;
        // the tile whose sums come next: its place, and its factors on their way
        int64_t first = 0, out_n = 0;
        int left = 0;
        float xa[kHalf / 32], w = 0.f;
        auto open = [&](int64_t id) {
            if (id >= total) return;
            RowTile t;
            int n;
            place(id, t, n);
            left = min(t.rows - h * kHalf, kHalf);   // tokens of this half
            first = (int64_t)t.row0 + h * kHalf;
            out_n = (int64_t)n * 256 + rank * 128 + row;
            w = out_n < g.N ? g.ws[(int64_t)t.group * g.N + out_n] : 0.f;
#pragma unroll
            for (int i = 0; i < kHalf / 32; ++i) xa[i] = i * 32 + lane < left ? g.xs[first + i * 32 + lane] : 0.f;
        };
        // Up to two chunks are added in fp32: a sum of two integers of 24 bits is rounded as the integer is at the end.
        const bool floats = PARTS == 1 && chunks <= 2;
        int64_t id = pair, end = min(kb, kChunkBlocks);   // end: the k-block behind the next chunk, counted over all tiles
        int64_t tiles_left = tiles, owed_at = 0;
        int done = 0;                                     // k-blocks of the tile in chunks that were added
        uint32_t use = 0;
        bool ok = true, owed = false;                     // owed: a tile's sums are in registers, not yet stored
        int acc[kHalf];
#pragma unroll
        for (int i = 0; i < kHalf; ++i) acc[i] = 0;
        open(id);
        for (int64_t i = h; ok; i += 2) {
            while (ok) {
                // A chunk's sums are read before the second k-block behind it is converted: its MMAs wait for that.  (Before the first,
                // or as soon as they are there: 5 to 14% slower, since conversions then wait; before the third: 15%.)  A tile is
                // stored after two more, so that converted k-blocks are left for the MMAs meanwhile.
                const bool due = tiles_left > 0 && (end + 2 <= i || i >= blocks);
                if (PARTS == 1 && owed && (due || i >= owed_at || i >= blocks)) {
                    owed = false;
#pragma unroll
                    for (int j = 0; j < kHalf / 32; ++j) xs[j * 32 + lane] = xa[j];
                    __syncwarp();
                    if (out_n < g.N && left > 0) {
                        auto value = [&](int j) { return (floats ? __int_as_float(acc[j]) : (float)acc[j]) * xs[j] * w; };
                        if (g.out_f32) {
                            float *out = static_cast<float *>(g.out) + first * g.N + out_n;
#pragma unroll
                            for (int j = 0; j < kHalf; ++j, out += g.N)
                                if (j < left) *out = value(j);
                        } else {
                            uint16_t *out = static_cast<uint16_t *>(g.out) + first * g.N + out_n;
#pragma unroll
                            for (int j = 0; j < kHalf; ++j, out += g.N)
                                if (j < left) *out = f32_to_bf16_bits(value(j));
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < kHalf; ++j) acc[j] = 0;
                    id += n_pairs;
                    open(id);
                    continue;
                }
                if (!due) break;
                if (left > 0) {   // (a tile of up to kHalf tokens has no second half)
                    ok = wait_all(smem_u32(&ctl->dfull[h]), use & 1u, abort_flag, g);
                    if (!ok) break;
                    ++use;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kHalf; c += 32) {
                        uint32_t v[32];
                        tmem_ld32(src + c, v);
                        tmem_ld_wait();
                        if (c + 32 == kHalf) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) arrive_cluster_relaxed(dempty);
                        }
                        if (floats) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                acc[c + j] = __float_as_int(__int_as_float(acc[c + j]) + __uint_as_float(v[j]));
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) acc[c + j] += __float2int_rn(__uint_as_float(v[j]));
                        }
                    }
                }
                done += min(kb - done, kChunkBlocks);
                if (done == kb) {
                    owed = true;
                    owed_at = i + 4;
                    done = 0;
                    --tiles_left;
                }
                end += min(kb - done, kChunkBlocks);
            }
            if (!ok || i >= blocks) break;
            const int stage = (int)(i % kStages), a = (int)(i % kSlots);
            // (in this order: the slot's wait says that the stage's k-block before this one has landed)
            ok = wait_all(smem_u32(&ctl->aempty[a]), ((uint32_t)(i / kSlots) & 1u) ^ 1u, abort_flag, g) &&
                 wait_all(smem_u32(&ctl->wfull[stage]), (uint32_t)(i / kStages) & 1u, abort_flag, g);
            if (!ok) break;
            tc_fence_after();
            convert_rows(ring + (size_t)stage * kStage, row, tmem_a + (uint32_t)(a * kATmem) + lanes);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(map_to_rank(smem_u32(&ctl->afull[a]), first_rank));
        }
        __syncwarp();
        if constexpr (PARTS > 1) {
            // Either pair finishes half of the token columns of either half: it sends its sums of the others to the CTA with the
            // same weight rows, [half][group of four columns][row], in the rings.
            constexpr int kMine = kHalf / 2;
            int4 *red = reinterpret_cast<int4 *>(ring);
            static_assert(2 * (kMine / 4) * 128 * 16 <= kStages * kStage, "exchange");
            cluster_sync();   // every ring of the cluster is idle
#pragma unroll
            for (int c = 0; c < kMine; c += 4) {
                const int4 v = part == 0 ? make_int4(acc[kMine + c], acc[kMine + c + 1], acc[kMine + c + 2], acc[kMine + c + 3])
                                         : make_int4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
                st_cluster_s32x4(map_to_rank(smem_u32(red + (h * (kMine / 4) + c / 4) * 128 + row), in_cluster ^ 2u), v);
            }
#pragma unroll
            for (int j = 0; j < kHalf / 32; ++j) xs[j * 32 + lane] = xa[j];
            cluster_sync();
            if (ok && tiles > 0 && out_n < g.N) {
                const int from = part * kMine;
                const int64_t at = (first + from) * g.N + out_n;
                float *out = static_cast<float *>(g.out) + at;
                uint16_t *out16 = static_cast<uint16_t *>(g.out) + at;
#pragma unroll
                for (int c = 0; c < kMine; c += 4) {
                    const int4 v = red[(h * (kMine / 4) + c / 4) * 128 + row];
                    const int sum[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j, out += g.N, out16 += g.N) {
                        const int mine = part == 0 ? acc[c + j] : acc[kMine + c + j];
                        if (from + c + j < left) {
                            const float y = (float)(mine + sum[j]) * xs[from + c + j] * w;
                            if (g.out_f32)
                                *out = y;
                            else
                                *out16 = f32_to_bf16_bits(y);
                        }
                    }
                }
            }
            __syncwarp();
        }
    }

    // ---- teardown: every issued stage is released by the leader's MMA commit once its bytes (of both CTAs) have landed and been
    // used; after an abort the waits are bounded
    if (warp == 0 && lane == 0) {
        for (int64_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
            if (!mbar_wait_drain(smem_u32(&ctl->empty[i % kStages]), (uint32_t)((i / kStages) & 1),
                                 drain_limit_of(g.wait_limit_ns)))
                __nanosleep(200000);
    }
    if (warp == 1 && lane == 0 && leader) {
        tc_commit_pair_multicast(smem_u32(&ctl->drain), (uint16_t)(1u << first_rank));
        (void)mbar_wait_drain(smem_u32(&ctl->drain), 0, drain_limit_of(g.wait_limit_ns));
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

// Opts the kernel into its shared memory once per device.
template <int PARTS>
cudaError_t prepare() {
    static std::atomic<uint64_t> done;   // bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (done.load(std::memory_order_acquire) >> (dev & 63) & 1)) return e;
    // the hand-over of registers needs the ones it was written for
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, int8_pair_kernel<PARTS>)) != cudaSuccess) return e;
    if (at.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(int8_pair_kernel<PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e == cudaSuccess) done.fetch_or(1ull << (dev & 63), std::memory_order_acq_rel);
    return e;
}

// Clusters of two pairs that can be resident at once (0 on failure).
int resident_clusters() {
    static std::atomic<int> cache[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if ((n = cache[dev & 63].load()) > 0) return n;
    if (prepare<2>() != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(4);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 4;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, int8_pair_kernel<2>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    cache[dev & 63].store(n);
    return n;
}

template <int PARTS>
cudaError_t run(const CUtensorMap &tw, const CUtensorMap &tx, const Int8Gemm &g, int kb, int n_tiles_n, int64_t clusters, bool pdl,
                cudaStream_t s) {
    const cudaError_t e = prepare<PARTS>();
    if (e != cudaSuccess) return e;
    return launch_kernel(int8_pair_kernel<PARTS>, dim3((unsigned)(2 * PARTS * clusters)), kThreads, kSmem, pdl, 2 * PARTS, s, tw, tx, g,
                         kb, n_tiles_n);
}

}  // namespace

// Pairs that share a tile's k-blocks: two where every tile has a cluster of its own.  (us with one pair and two: 1024 x 2112 x 7168,
// 36 tiles, 47.2, 32.4; the swap-AB kernel takes 37.8.)
int int8_pair_parts(int64_t tiles, int kb) { return kb >= 8 && tiles <= resident_clusters() ? 2 : 1; }

int64_t int8_pair_tiles(const Int8Gemm &g) {
    return ((g.T + kTokens - 1) / kTokens + (g.offsets ? std::min<int64_t>(g.groups, g.T) : 0)) * ((g.N + 255) / 256);
}

mse_status launch_int8_pair(const Int8Gemm &g, int sm_count, bool pdl, cudaStream_t s) {
    CUtensorMap tw, tx;
    mse_status st = map_bytes(&tw, g.wq, g.groups * g.N, g.K, g.ldw, 128);
    if (st != MSE_OK) return st;
    if ((st = map_bytes(&tx, g.x16, g.T, g.K * 2, g.ldx16 * 2, kHalf / 2)) != MSE_OK) return st;
    const int kb = (int)((g.K + kInner - 1) / kInner), n_tiles_n = (int)((g.N + 255) / 256);
    const int64_t tiles = int8_pair_tiles(g);
    const cudaError_t e = int8_pair_parts(tiles, kb) == 2
                              ? run<2>(tw, tx, g, kb, n_tiles_n, tiles, pdl, s)
                              : run<1>(tw, tx, g, kb, n_tiles_n, std::min<int64_t>(sm_count / 2, tiles), pdl, s);
    return e == cudaSuccess ? MSE_OK : MSE_ERR_CUDA;
}

}  // namespace sorted
}  // namespace mse
