// Routing of tokens to experts: scores, groups, the best top_k, their weights.
//
// One warp per token; lane l holds experts l, l + 32, ... in registers.  Everything after the
// one read of the logits stays in the warp.  The top_k-th largest of the 32 lanes' best keys bounds
// the top_k-th best key from below; the few keys that reach it are gathered, and each counts the
// ones before it: its rank is its place.  (Only where more than 32 reach it, by ties, is the best
// key drawn top_k times.)  What bounds it is the instructions of a warp, not the logits' bytes.
#include "common.cuh"
#include "launch.h"
#include "routed.h"

namespace mse {
namespace routed {
namespace {

constexpr int kRouteWarps = 8;
// the lowest finite bf16: a logit at or below it (both types' lowest values, -inf) or NaN closes
// its expert
constexpr float kClosedFrom = -3.3895313892515355e38f;

// Order-preserving map of a float to an unsigned integer; every finite float maps above 0.
__device__ __forceinline__ uint32_t float_key(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);   // -0 counts as 0
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t k) {
    return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const RouteParams &p, int64_t i) {
    return BF16 ? bf16_bits_to_f32(__ldg(static_cast<const uint16_t *>(p.logits) + i))
                : __ldg(static_cast<const float *>(p.logits) + i);
}

// Bit g * lanes for each group g that stays: the topk_group largest values, equal ones to the lower group.
// keys: this warp's in shared memory, group g's from g * pitch on (a pitch of `lanes` more than the group, so that
// the lanes of neighbouring groups read different banks).
__device__ __forceinline__ uint32_t best_groups(const RouteParams &p, const uint32_t *keys, int pitch, int lanes,
                                                int lane) {
    const int g = lane >> (31 - __clz(lanes)), r = lane & (lanes - 1);   // lanes: a power of two
    uint32_t k1 = 0, k2 = 0;   // the two best keys of the group
    if (g < p.n_group) {
#pragma unroll 4
        for (int i = r; i < p.group_size; i += lanes) {
            const uint32_t k = keys[g * pitch + i];
            k2 = max(k2, min(k, k1));
            k1 = max(k1, k);
        }
    }
    for (int d = 1; d < lanes; d <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(~0u, k1, d), o2 = __shfl_xor_sync(~0u, k2, d);
        k2 = max(max(k2, o2), min(k1, o1));
        k1 = max(k1, o1);
    }
    uint32_t value = k1;
    if (p.group_top == 2 && k2 != 0) value = float_key(__fadd_rn(key_float(k1), key_float(k2)));
    if (r != 0 || g >= p.n_group) value = 0;
    uint32_t kept = 0;
    for (int j = 0; j < p.topk_group; ++j) {
        const uint32_t m = __reduce_max_sync(~0u, value);
        if (m == 0) break;   // the others have no open expert
        const uint32_t holders = __ballot_sync(~0u, value == m), first = holders & (0u - holders);
        kept |= first;
        if (first >> lane & 1u) value = 0;
    }
    return kept;
}

__device__ __forceinline__ float warp_fmax(float v) {   // no lane holds a NaN
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// a / b to nearest, with inv = 1 / b to nearest: one residual step makes the product exact to the last
// bit (Markstein); tiny quotients, whose residual could be cut off, take the division itself.
__device__ __forceinline__ float quotient(float a, float b, float inv) {
    if (a < 1e-30f) return __fdiv_rn(a, b);
    const float q = __fmul_rn(a, inv);
    return fmaf(fmaf(-b, q, a), inv, q);
}

template <int VPL, bool BF16>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteParams p) {
    extern __shared__ uint32_t route_smem[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    // keys, experts and scores of up to 32 candidates, then (groups) the keys of all experts
    uint32_t *mine = route_smem + (size_t)warp * p.smem_words;
    uint32_t *cand_key = mine, *cand_id = mine + 32, *all_keys = mine + 96;
    float *cand_score = reinterpret_cast<float *>(mine + 64);
    const int lanes = p.group_lanes, pitch = p.group_size + lanes;
    pdl_wait();
    float bias[VPL];
    int shift[VPL];   // g * lanes of the expert's group g: its bit among the kept ones
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = i * 32 + lane;
        bias[i] = p.bias && e < p.E ? __ldg(p.bias + e) : 0.f;
        shift[i] = (int)((uint32_t)e * (uint32_t)p.group_magic >> 20) * lanes;   // e / group_size
    }
    for (int64_t t = (int64_t)blockIdx.x * warps + warp; t < p.T; t += (int64_t)gridDim.x * warps) {
        float score[VPL];
        uint32_t key[VPL];   // 0: closed
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = i * 32 + lane;
            score[i] = e < p.E ? load_logit<BF16>(p, t * p.ld + e) : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool open = score[i] > kClosedFrom;
            key[i] = open ? 1u : 0u;
            score[i] = open ? score[i] : -INFINITY;
            top = fmaxf(top, score[i]);
        }
        if (p.sigmoid) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) score[i] = __frcp_rn(__fadd_rn(1.0f, expf(-score[i])));
        } else {
            top = warp_fmax(top);
            // The sum as if rounded once, whatever the order: each term e <= 1 is split into a
            // multiple of 2^-14 (at most 1024 of them add up exactly, here and as integers) and a
            // remainder of at most 2^-15, summed per lane in fp32 and over the lanes in units of 2^-36:
            // its errors lie 2^-12 below the last bit of the total.
            float high = 0.f, low = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                score[i] = key[i] ? expf(__fsub_rn(score[i], top)) : 0.f;
                const float h = __fsub_rn(__fadd_rn(score[i], 512.f), 512.f);
                high += h;
                low += __fsub_rn(score[i], h);
            }
            const int hi = __reduce_add_sync(~0u, __float2int_rn(high * 0x1p14f));
            const int lo = __reduce_add_sync(~0u, __float2int_rn(low * 0x1p36f));
            const float sum = fmaxf(fmaf((float)lo, 0x1p-36f, (float)hi * 0x1p-14f), 1e-30f), inv = __frcp_rn(sum);
#pragma unroll
            for (int i = 0; i < VPL; ++i) score[i] = quotient(score[i], sum, inv);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i]) key[i] = float_key(__fadd_rn(score[i], bias[i]));   // (x + 0 is x)
        if (p.n_group > 1) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i * 32 + lane < p.E) all_keys[shift[i] + i * 32 + lane] = key[i];   // g * pitch + e % group_size
            __syncwarp();
            const uint32_t kept = best_groups(p, all_keys, pitch, lanes, lane);
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (!(kept >> (shift[i] & 31) & 1u)) key[i] = 0;
        }
        // lower bound of the top_k-th best key: as many lanes hold one at least as large
        uint32_t lane_best = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) lane_best = max(lane_best, key[i]);
        uint32_t bound = 0;
        for (int j = 0; j < p.top_k; ++j) {
            bound = __reduce_max_sync(~0u, lane_best);
            if (bound == 0) break;
            const uint32_t holders = __ballot_sync(~0u, lane_best == bound);
            if ((holders & (0u - holders)) >> lane & 1u) lane_best = 0;
        }
        bound = max(bound, 1u);   // fewer lanes than top_k: every open key
        int n = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool in = key[i] >= bound;
            const uint32_t who = __ballot_sync(~0u, in);
            const int at = n + __popc(who & ((1u << lane) - 1u));
            if (in && at < 32) {
                cand_key[at] = key[i];
                cand_id[at] = i * 32 + lane;
                cand_score[at] = score[i];
            }
            n += __popc(who);
        }
        __syncwarp();
        int id = -1;   // lane j: the j-th best
        float w = 0.f;
        if (n <= 32) {
            const uint32_t k = lane < n ? cand_key[lane] : 0u;
            const uint32_t e = lane < n ? cand_id[lane] : 0u;
            const float sc = lane < n ? cand_score[lane] : 0.f;
            int rank = 0;   // candidates lie in the order of their experts: of equal keys the earlier is the better
            for (int j = 0; j < n; ++j) {
                const uint32_t o = cand_key[j];
                rank += o > k || (o == k && j < lane) ? 1 : 0;
            }
            __syncwarp();
            if (lane < n) {   // every candidate to its place
                cand_id[rank] = e;
                cand_score[rank] = sc;
            }
            __syncwarp();
            if (lane < n && lane < p.top_k) {
                id = (int)cand_id[lane];
                w = cand_score[lane];
            }
            __syncwarp();   // the next token's candidates come after these reads
        } else {
            for (int j = 0; j < p.top_k; ++j) {
                uint32_t best = 0;
                int at = 0;
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (key[i] > best) { best = key[i]; at = i; }
                const uint32_t m = __reduce_max_sync(~0u, best);
                if (m == 0) break;
                const uint32_t e = __reduce_min_sync(~0u, best == m ? (uint32_t)(at * 32 + lane) : ~0u);
                float sc = 0.f;
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if ((uint32_t)(i * 32 + lane) == e) { key[i] = 0; sc = score[i]; }
                sc = __shfl_sync(~0u, sc, e % 32);
                if (lane == j) { id = (int)e; w = sc; }
            }
        }
        if (p.renormalise) {
            float total = w;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(~0u, total, d);
            if (total > 0.f) w = __fdiv_rn(w, total);
        }
        if (lane < p.top_k) {
            p.ids[t * p.top_k + lane] = id;
            p.weights[t * p.top_k + lane] = w * p.scale;
        }
        }
    }

    template <int VPL>
    cudaError_t launch_vpl(RouteParams p, int sm_count, bool pdl, cudaStream_t s) {
        // a few tokens: one warp per CTA, so that they run on as many SMs
        const int warps = p.T >= 1024 ? kRouteWarps : 1;
        p.group_lanes = p.n_group > 16 ? 1 : p.n_group > 8 ? 2 : p.n_group > 4 ? 4 : p.n_group > 2 ? 8 : 16;
        p.group_magic = ((1 << 20) + p.group_size - 1) / p.group_size;   // exact for e < 1024
        p.smem_words = 96 + (p.n_group > 1 ? p.n_group * (p.group_size + p.group_lanes) : 0);
        const size_t smem = (size_t)p.smem_words * 4 * warps;
        // a warp keeps its experts' biases and groups from token to token
        const dim3 grid((unsigned)std::min<int64_t>((p.T + warps - 1) / warps, (int64_t)sm_count * 8));
        return p.bf16_logits ? launch_kernel(route_kernel<VPL, true>, grid, warps * 32, smem, pdl, 1, s, p)
                             : launch_kernel(route_kernel<VPL, false>, grid, warps * 32, smem, pdl, 1, s, p);
    }

    }  // namespace

    cudaError_t launch_route(const RouteParams &p, int sm_count, bool pdl, cudaStream_t s) {
        switch ((p.E + 31) / 32) {
            case 1: return launch_vpl<1>(p, sm_count, pdl, s);
            case 2: return launch_vpl<2>(p, sm_count, pdl, s);
            case 3: return launch_vpl<3>(p, sm_count, pdl, s);
            case 4: return launch_vpl<4>(p, sm_count, pdl, s);
            case 5: return launch_vpl<5>(p, sm_count, pdl, s);
            case 6: return launch_vpl<6>(p, sm_count, pdl, s);
            case 7: case 8: return launch_vpl<8>(p, sm_count, pdl, s);
            case 9: case 10: return launch_vpl<10>(p, sm_count, pdl, s);
            case 11: case 12: return launch_vpl<12>(p, sm_count, pdl, s);
            case 13: case 14: case 15: case 16: return launch_vpl<16>(p, sm_count, pdl, s);
            default: return launch_vpl<32>(p, sm_count, pdl, s);
        }
    }

    }  // namespace routed
    }  // namespace mse
