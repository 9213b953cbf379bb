// Routing of tokens to experts: scores, groups, the best top_k, their weights.
//
// One warp per token; lane l holds experts l, l + 32, ... in registers.  Everything after the
// one read of the logits stays in the warp.  What bounds it is a warp's instructions, not the
// logits' bytes, so the exact score (an accurate exponential and division) is computed for a few
// experts only:
//   - every expert gets its choice to about 2^-18 by the fast exponential and reciprocal;
//   - the top_k-th largest of the 32 lanes' best ones bounds the top_k-th best from below, and
//     the experts within twice the error of that bound, a few more than top_k, are gathered;
//   - each of them gets its exact choice and counts the ones before it: its rank is its place.
// Where more than 32 are that near, the exact choices of all are drawn from top_k times.  With
// groups the groups' values need exact choices, so all are exact from the start.
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
constexpr float kLowest = -3.4028234663852886e38f;   // of fp32: a bias may bring a choice down to it

template <bool BF16>
__device__ __forceinline__ float load_logit(const RouteParams &p, int64_t i) {
    return BF16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(p.logits)[i])
                : static_cast<const float *>(p.logits)[i];
}

__device__ __forceinline__ float warp_fmax(float v) {
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// a / b to nearest, with inv = 1 / b to nearest: one residual step makes the product exact to the last
// bit (Markstein), 0 included.  Not for tiny a, whose residual is cut off: they take the division itself.
__device__ __forceinline__ float quotient(float a, float b, float inv) {
    const float q = __fmul_rn(a, inv);
    return fmaf(fmaf(-b, q, a), inv, q);
}
__device__ __forceinline__ bool is_tiny(float a) { return a < 1e-30f && a > 0.f; }

// Bit g * lanes for each group g that stays: the topk_group largest values, equal ones to the lower group.
// choices: this warp's in shared memory (-inf: closed), group g's from g * pitch on (a pitch of `lanes` more than
// the group, so that the lanes of neighbouring groups read different banks).
__device__ __forceinline__ uint32_t best_groups(const RouteParams &p, const float *choices, int pitch, int lanes,
                                                int lane) {
    const int g = lane >> (31 - __clz(lanes)), r = lane & (lanes - 1);   // lanes: a power of two
    float c1 = -INFINITY, c2 = -INFINITY;                                // the group's two best
    if (g < p.n_group) {
#pragma unroll 4
        for (int i = r; i < p.group_size; i += lanes) {
            const float c = choices[g * pitch + i];
            c2 = fmaxf(c2, fminf(c, c1));
            c1 = fmaxf(c1, c);
        }
    }
    for (int d = 1; d < lanes; d <<= 1) {
        const float o1 = __shfl_xor_sync(~0u, c1, d), o2 = __shfl_xor_sync(~0u, c2, d);
        c2 = fmaxf(fmaxf(c2, o2), fminf(c1, o1));
        c1 = fmaxf(c1, o1);
    }
    // (two lowest choices add up to -inf, but a group that has any comes before one that has none)
    float value = p.group_top == 2 && c2 > -INFINITY ? fmaxf(__fadd_rn(c1, c2), kLowest) : c1;
    if (r != 0 || g >= p.n_group) value = -INFINITY;
    uint32_t kept = 0;
    for (int j = 0; j < p.topk_group; ++j) {
        const float m = warp_fmax(value);
        if (m == -INFINITY) break;   // the others have no open expert
        const uint32_t holders = __ballot_sync(~0u, value == m), first = holders & (0u - holders);
        kept |= first;
        if (first >> lane & 1u) value = -INFINITY;
    }
    return kept;
}

// A token with an infinite logit under softmax: e^(l - max) / sum is NaN for every open expert.  Equal choices, so the lowest
// open experts of the lowest groups with one, and weights of NaN: an overflow before the router shows in what follows.
// Bit i of `open`: expert i * 32 + lane.
__device__ __forceinline__ void undefined_scores(const RouteParams &p, int64_t t, uint32_t open, int per_lane, int lane) {
    int id = -1, n = 0, groups = 0, group = -1;
#pragma unroll 1
    for (int i = 0; i < per_lane && n < p.top_k; ++i) {
        for (uint32_t which = __ballot_sync(~0u, open >> i & 1u); which != 0 && n < p.top_k; which &= which - 1u) {
            const int e = i * 32 + __ffs(which) - 1;
            if (e / p.group_size != group) {
                group = e / p.group_size;
                if (++groups > p.topk_group) {
                    n = p.top_k;   // no more groups
                    break;
                }
            }
            if (lane == n) id = e;
            ++n;
        }
    }
    if (lane < p.top_k) {
        p.ids[t * p.top_k + lane] = id;
        p.weights[t * p.top_k + lane] = id >= 0 ? __int_as_float(0x7FC00000) : 0.f;
    }
}

template <int VPL, bool BF16, bool GROUPS>
__global__ void __launch_bounds__(kRouteWarps * 32, VPL <= 8 ? 5 : VPL <= 16 ? 4 : 2) route_kernel(const RouteParams p) {
    extern __shared__ float route_smem[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    // up to 32 candidates, then (groups) the choices and the scores of all experts
    float *cand_choice = route_smem + (size_t)warp * p.smem_words, *cand_score = cand_choice + 32;
    int *cand_id = reinterpret_cast<int *>(cand_choice + 64);
    float *all_choices = cand_choice + 96;
    const int lanes = p.group_lanes, pitch = p.group_size + lanes;
    float *all_scores = all_choices + p.n_group * pitch;
    pdl_wait();
    // Up to 384 experts a warp keeps their biases and groups from token to token; with more, warps on the SM
    // are worth more than these registers (23405 x 448 in 8 groups 45 us, 98 with them).
    constexpr bool KEEP = VPL <= 12;
    float bias[KEEP ? VPL : 1] = {};
    int shift[KEEP && GROUPS ? VPL : 1] = {};   // g * lanes of the expert's group g: its bit among the kept ones
    auto load_bias = [&](int i) { return p.bias && i * 32 + lane < p.E ? p.bias[i * 32 + lane] : 0.f; };
    auto find_shift = [&](int i) { return (int)((uint32_t)(i * 32 + lane) * (uint32_t)p.group_magic >> 20) * lanes; };
    if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            bias[i] = load_bias(i);
            if constexpr (GROUPS) shift[i] = find_shift(i);
        }
    }
    auto bias_of = [&](int i) { return KEEP ? bias[KEEP ? i : 0] : load_bias(i); };
    auto shift_of = [&](int i) { return KEEP && GROUPS ? shift[KEEP && GROUPS ? i : 0] : find_shift(i); };
    for (int64_t t = (int64_t)blockIdx.x * warps + warp; t < p.T; t += (int64_t)gridDim.x * warps) {
        float v[VPL];        // logit (-inf: closed), then the softmax's term, then the choice
        uint32_t open = 0;   // bit i
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = i * 32 + lane;
            v[i] = e < p.E ? load_logit<BF16>(p, t * p.ld + e) : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            v[i] = v[i] > kClosedFrom ? v[i] : -INFINITY;
            open |= v[i] > -INFINITY ? 1u << i : 0u;
        }
        float top = -INFINITY, sum = 1.f, inv = 1.f;
        if (!p.sigmoid) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) top = fmaxf(top, v[i]);
            top = warp_fmax(top);
            if (top == INFINITY) {
                undefined_scores(p, t, open, VPL, lane);
                continue;
            }
            if (top == -INFINITY) top = 0.f;
            // The sum as if rounded once, whatever the order: each term e <= 1 is split into a
            // multiple of 2^-14 (at most 1024 of them add up exactly, here and as integers) and a
            // remainder of at most 2^-15, summed per lane in fp32 and over the lanes in units of 2^-36:
            // its errors lie 2^-12 below the last bit of the total.
            float high = 0.f, low = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                v[i] = expf(__fsub_rn(v[i], top));   // closed: 0
                const float h = __fsub_rn(__fadd_rn(v[i], 512.f), 512.f);
                high += h;
                low += __fsub_rn(v[i], h);
            }
            const int hi = __reduce_add_sync(~0u, __float2int_rn(high * 0x1p14f));
            const int lo = __reduce_add_sync(~0u, __float2int_rn(low * 0x1p36f));
            sum = fmaxf(fmaf((float)lo, 0x1p-36f, (float)hi * 0x1p-14f), 1e-30f);
            inv = __frcp_rn(sum);
        }
        auto divided = [&](float e) { return is_tiny(e) ? __fdiv_rn(e, sum) : quotient(e, sum, inv); };
        auto score_of = [&](float logit) {   // exact
            return p.sigmoid ? __frcp_rn(__fadd_rn(1.0f, expf(-logit)))
                             : divided(expf(__fsub_rn(logit, top)));
        };
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            float c;
            if constexpr (GROUPS) {
                const float sc = p.sigmoid ? __frcp_rn(__fadd_rn(1.0f, expf(-v[i]))) : divided(v[i]);
                if (i * 32 + lane < p.E) all_scores[i * 32 + lane] = sc;
                c = __fadd_rn(sc, bias_of(i));
            } else
                c = p.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-v[i])) + bias_of(i)
                              : fmaf(v[i], inv, bias_of(i));
            v[i] = (open >> i & 1u) && c >= -INFINITY ? c : -INFINITY;   // (a NaN of the bias is no choice)
        }
        if constexpr (GROUPS) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i * 32 + lane < p.E)
                    all_choices[shift_of(i) + i * 32 + lane] = v[i];   // g * pitch + e % group_size
            __syncwarp();
            const uint32_t kept = best_groups(p, all_choices, pitch, lanes, lane);
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (!(kept >> (shift_of(i) & 31) & 1u)) v[i] = -INFINITY;
        }
        // as many lanes as top_k hold a choice at least as large as the bound
        float lane_best = -INFINITY, bound = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) lane_best = fmaxf(lane_best, v[i]);
        for (int j = 0; j < p.top_k; ++j) {
            bound = warp_fmax(lane_best);
            if (bound == -INFINITY) break;
            const uint32_t holders = __ballot_sync(~0u, lane_best == bound);
            if ((holders & (0u - holders)) >> lane & 1u) lane_best = -INFINITY;
        }
        if constexpr (!GROUPS) {
            // twice the error of a fast choice: 2^-18 of the score (an exponent of up to 88 costs the fast
            // exponential 2^-18), the sum with the bias 2^-22 of the result
            const float slack = fabsf(bound) * 0x1p-16f + (p.bias ? 0x1p-17f : 0.f);
            bound = !p.bias && bound < 1e-30f ? kLowest : bound - slack;   // (tiny scores: all of them)
        }
        bound = fmaxf(bound, kLowest);   // fewer lanes than top_k (or NaN: infinite choices): every open expert
        uint32_t in = 0;                     // bit i: candidate
#pragma unroll
        for (int i = 0; i < VPL; ++i) in |= v[i] >= bound ? 1u << i : 0u;
        int n = 0;
        for (;;) {
            const uint32_t who = __ballot_sync(~0u, in != 0);
            if (who == 0) break;
            const int at = n + __popc(who & ((1u << lane) - 1u));
            if (in != 0 && at < 32) cand_id[at] = (__ffs(in) - 1) * 32 + lane;
            in &= in - 1u;
            n += __popc(who);
        }
        __syncwarp();
        int id = -1;   // lane j: the j-th best
        float w = 0.f;
        if (n <= 32) {
            int e = 0;
            float sc = 0.f, c = -INFINITY;
            if (lane < n) {
                e = cand_id[lane];
                sc = GROUPS ? all_scores[e] : score_of(load_logit<BF16>(p, t * p.ld + e));
                c = p.bias ? __fadd_rn(sc, p.bias[e]) : sc;
                cand_choice[lane] = c;
            }
            __syncwarp();
            int rank = 0;
            for (int j = 0; j < n; ++j) {
                const float o = cand_choice[j];
                rank += o > c || (o == c && cand_id[j] < e) ? 1 : 0;
            }
            __syncwarp();
            if (lane < n) {   // every candidate to its place
                cand_id[rank] = e;
                cand_score[rank] = sc;
            }
            __syncwarp();
            if (lane < n && lane < p.top_k) {
                id = cand_id[lane];
                w = cand_score[lane];
            }
            __syncwarp();   // the next token's candidates come after these reads
        } else {
            if constexpr (!GROUPS) {
#pragma unroll 1
                for (int i = 0; i < VPL; ++i) {
                    const int x = i * 32 + lane;
                    float c = -INFINITY;
                    if (open >> i & 1u)
                        c = __fadd_rn(score_of(load_logit<BF16>(p, t * p.ld + x)), p.bias ? p.bias[x] : 0.f);
#pragma unroll
                    for (int u = 0; u < VPL; ++u)
                        if (u == i) v[u] = c;
                }
            }
            for (int j = 0; j < p.top_k; ++j) {
                float best = -INFINITY;
                int at = 0;
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (v[i] > best) { best = v[i]; at = i; }
                const float m = warp_fmax(best);
                if (m == -INFINITY) break;
                const uint32_t e = __reduce_min_sync(~0u, best == m ? (uint32_t)(at * 32 + lane) : ~0u);
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if ((uint32_t)(i * 32 + lane) == e) v[i] = -INFINITY;
                if (lane == j) id = (int)e;
            }
            if (id >= 0) w = score_of(load_logit<BF16>(p, t * p.ld + id));
            __syncwarp();   // (groups: the next token's scores come after the reads of this one's)
        }
        if (p.renormalise) {
            float total = w;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(~0u, total, d);
            if (total > 0.f) w = __fdiv_rn(w, total);
        }
        if (lane < p.top_k) {
            p.ids[t * p.top_k + lane] = id;
            p.weights[t * p.top_k + lane] = id >= 0 ? w * p.scale : 0.f;
        }
    }
}

template <int VPL>
cudaError_t launch_vpl(RouteParams p, int sm_count, bool pdl, cudaStream_t s) {
    // a few tokens: one warp per CTA, so that they run on as many SMs
    const int warps = p.T >= 1024 ? kRouteWarps : 1;
    p.group_lanes = p.n_group > 16 ? 1 : p.n_group > 8 ? 2 : p.n_group > 4 ? 4 : p.n_group > 2 ? 8 : 16;
    p.group_magic = ((1 << 20) + p.group_size - 1) / p.group_size;   // exact for e < 1024
    p.smem_words = 96 + (p.n_group > 1 ? p.n_group * (p.group_size + p.group_lanes) + p.E : 0);
    const size_t smem = (size_t)p.smem_words * 4 * warps;   // at most 70 KB
    if (smem > 48 * 1024) {   // groups of over 700 experts
        const cudaError_t e = p.bf16_logits ? cudaFuncSetAttribute(route_kernel<VPL, true, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)
                                            : cudaFuncSetAttribute(route_kernel<VPL, false, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    // as many CTAs as can be resident, and then some
    const dim3 grid((unsigned)std::min<int64_t>((p.T + warps - 1) / warps, (int64_t)sm_count * 8));
    const int threads = warps * 32;
    if (p.n_group > 1)
        return p.bf16_logits ? launch_kernel(route_kernel<VPL, true, true>, grid, threads, smem, pdl, 1, s, p)
                             : launch_kernel(route_kernel<VPL, false, true>, grid, threads, smem, pdl, 1, s, p);
    return p.bf16_logits ? launch_kernel(route_kernel<VPL, true, false>, grid, threads, smem, pdl, 1, s, p)
                         : launch_kernel(route_kernel<VPL, false, false>, grid, threads, smem, pdl, 1, s, p);
}

}  // namespace

// Experts a lane.  Beside the powers of two, classes for 129 to 192, 257 to 384 and 385 to 448 experts, whose unused registers and
// steps cost most (us with them and with the next power of two: 65536 x 160 in 8 groups 57.2, 75.7; 65536 x 192 67.7, 80.5;
// 32768 x 384 in 8 groups 51.8, 67.4; 23405 x 448 45.4, 49.3; 8192 x 160 without groups 6.8, 7.8; 192 8.0, 8.6; 384 9.9,
// 10.7; 448 10.1, 10.6).  Other numbers take the next class (8192 x 320 9.6, 8192 x 96 6.4, like 128), from 513 on the
// one of 1024.
cudaError_t launch_route(const RouteParams &p, int sm_count, bool pdl, cudaStream_t s) {
    switch ((p.E + 31) / 32) {
        case 1: return launch_vpl<1>(p, sm_count, pdl, s);
        case 2: return launch_vpl<2>(p, sm_count, pdl, s);
        case 3: case 4: return launch_vpl<4>(p, sm_count, pdl, s);
        case 5: return launch_vpl<5>(p, sm_count, pdl, s);
        case 6: return launch_vpl<6>(p, sm_count, pdl, s);
        case 7: case 8: return launch_vpl<8>(p, sm_count, pdl, s);
        case 9: case 10: case 11: case 12: return launch_vpl<12>(p, sm_count, pdl, s);
        case 13: case 14: return launch_vpl<14>(p, sm_count, pdl, s);
        case 15: case 16: return launch_vpl<16>(p, sm_count, pdl, s);
        default: return launch_vpl<32>(p, sm_count, pdl, s);
    }
}

}  // namespace routed
}  // namespace mse
