// C-ABI entry points of the routed-expert operators: argument validation (before any CUDA call),
// workspace carving and kernel choice.
#include <algorithm>
#include <cstring>

#include "device.h"
#include "routed.h"

using namespace mse;
using namespace mse::routed;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;     // rows and columns: indexes of tiles stay in 32 bits
constexpr int64_t kMaxInner = (int64_t)1 << 22;
constexpr int64_t kMaxPitch = (int64_t)1 << 32;

size_t up256(size_t v) { return (v + 255) / 256 * 256; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned256(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
bool disjoint(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x + (uintptr_t)a_bytes <= y || y + (uintptr_t)b_bytes <= x;
}
mse_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MSE_OK : MSE_ERR_CUDA; }

// x in 8 bits and its scales
struct LinearWs {
    size_t q_off, s_off, total;
};
LinearWs linear_ws(int64_t T, int64_t K) {
    LinearWs w;
    w.q_off = 0;
    w.s_off = up256((size_t)T * (size_t)pad16(K));
    w.total = w.s_off + up256((size_t)T * (size_t)blocks_of(K) * 4);
    return w;
}

mse_status check_matmul(const void *xq, int64_t ldx, const void *xs, const void *wq, int64_t ldw, const void *ws,
                        int64_t T, int64_t N, int64_t K, const void *out, mse_dtype dtype, int64_t capacity) {
    if (!xq || !xs || !wq || !ws || !out || T <= 0 || N <= 0 || K <= 0 || ldx < K || ldw < K ||
        ldx > kMaxPitch || ldw > kMaxPitch ||
        (dtype != MSE_BF16 && dtype != MSE_F32) || T > kMaxRows || N > kMaxInner || K > kMaxInner)
        return MSE_ERR_INVALID_ARG;
    return capacity < T * N ? MSE_ERR_GEOMETRY : MSE_OK;
}

// Token rows of a tile: 16, 32 and 64 take the swap-AB kernel, 256 the CTA-pair kernel.
//
// Plain product: the kernel that is expected to take less time, in units of 0.01 us.  A CTA pair (half as many as SMs)
// spends 0.41 us on a k-block of 256 x 256, two swap-AB CTAs on an SM 0.54 us on one of 128 x 64 each; a split
// tile's exchange takes 2.5 us in the swap-AB kernel, 4 or 6 in the pair's, which starts 1.3 us later (us, pair and swap-AB:
// 256 x 7168 x 6144 18.6, 26.4; 128 x 12288 x 7168 27.1, 29.9; 512 x 2112 x 7168 17.8, 19.4; 320 x 2112 x 7168 17.7, 15.5;
// 64 x 12288 x 7168 26.3, 19.3; 128 x 4000 x 1000 9.0, 8.0; 1024 x 700 x 3000 13.6, 11.4).
int plain_tile_rows(int64_t T, int64_t N, int64_t K, int sm_count) {
    if (T <= 32) return T <= 16 ? 16 : 32;
    const int64_t kb = blocks_of(K), cols = blocks_of(N) * ((T + 63) / 64), pairs = ((T + 255) / 256) * ((N + 255) / 256);
    const int64_t cp = cols_parts(cols, (int)kb, 64, BLOCK_BF16, sm_count), pp = pair_parts(pairs, (int)kb);
    const int64_t cols_waves = (cols * cp + sm_count - 1) / sm_count, pair_waves = (pairs * pp + sm_count / 2 - 1) / (sm_count / 2);
    const int64_t cols_time = cols_waves * kb * 27 / cp + (cp > 1 ? 250 : 0);
    const int64_t pair_time = pair_waves * kb * 41 / pp + (pp == 4 ? 600 : pp == 2 ? 400 : 0) + 130;
    return pair_time < cols_time ? 256 : 64;
}
// Experts, by the rows expected of each, if all pairs were this rank's: the call does not know how many experts there are
// in all, and a rank that holds some of them gets larger tiles than its rows ask for (32 of 128 experts of 7168 x 2048 with
// 256 tokens, 16 rows each, 309 us, 280 with tiles of 16; 32 of 256, 8 rows, 306, 253; with 128 tokens 258, 230).  One bound
// between 32 and 256 for all sizes lies between what small and large experts would have (us with tiles of 16, 32 and 256; 32 experts of
// 7168 x 2048: 16 rows 247, 248, 313; 32 rows 311, 279, 322; 40 rows 371, 332, 327; 48 rows 407, 345, 332; 8 of 2048 x 1536:
// 16 rows 26, 27, 41; 48 rows 48, 36, 45; 64 rows 54, 42, 46; 80 rows 60, 53, 46; half of 64 experts of 1000 x 500, 50 rows
// 35, 32, 40; tiles of 64 and 128 were never the fastest).
int expert_tile_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 56 ? 32 : 256; }

mse_status run_product(BlockGemm g, bool tensorcore, const DeviceView &d, cudaStream_t s) {
    g.wait_limit_ns = wait_limit_ns();
    g.err = d.err;
    if (!tensorcore) return from_cuda(launch_block_simt(g, pdl_enabled(), s));
    if (g.tile_rows == 256) return launch_block_pair(g, d.sm_count, pdl_enabled(), s);
    return launch_block_cols(g, d.sm_count, pdl_enabled(), s);
}

BlockGemm plain_product(const uint8_t *xq, int64_t ldx, const float *xs, const uint8_t *wq, int64_t ldw,
                        const float *ws, int64_t T, int64_t N, int64_t K, void *out, mse_dtype dtype, int sm_count) {
    BlockGemm g;
    std::memset(&g, 0, sizeof g);
    g.T = T;
    g.tile_rows = plain_tile_rows(T, N, K, sm_count);
    g.xq = xq; g.ldx = ldx; g.xs = xs;
    g.wq = wq; g.ldw = ldw; g.ws = ws;
    g.N = N; g.K = K; g.kb = (int)blocks_of(K);
    g.groups = 1;
    g.w_group_rows = N;
    g.epi = dtype == MSE_F32 ? BLOCK_F32 : BLOCK_BF16;
    g.out = out; g.ldo = N;
    return g;
}

// One launch, whose kernel rounds the tokens itself, up to 8 tokens of a small weight: called one after another it saves the
// host a launch, and in a graph the two come to the same; every CTA rounds all tokens, which larger weights pay for.  (us with
// one launch and with two, called in a row, and in a graph with the weights from memory: 3 x 904 x 966 6.3, 8.7 and 5.1, 5.2;
// 8 x 1024 x 1024 6.1, 8.5 and 5.6, 5.4; 1 x 576 x 7168 7.3, 8.7 and 7.4, 7.6; 1 x 2112 x 7168 9.0, 9.2 and 8.9, 8.9;
// 8 x 4096 x 4096 9.7, 10.0 and 9.9, 10.0; beyond the bound 8 x 7168 x 6144 13.3, 13.3 and 13.6, 13.3; 1 x 12288 x 7168 18.6,
// 18.6 and 19.7, 19.3; 16 tokens of 1024 x 4096 8.4, 6.9.)
bool rounds_itself(int64_t T, int64_t N, int64_t K) { return T <= kRoundRows && N * K <= (int64_t)1 << 24; }

bool tc_operands(const void *xq, int64_t ldx, const void *wq, int64_t ldw) {
    return aligned16(xq) && aligned16(wq) && ldx % 16 == 0 && ldw % 16 == 0;
}

// ------------------------------------------------------------------ the experts' layer
// Up to this many pairs every CTA of the dispatch counts all ids itself.
constexpr int64_t kCountAllPairs = 4096;

// Tokens of a CTA of the dispatch: about as many CTAs as SMs, as far as a CTA's pairs reach.  (A constant, because the
// workspace's size, asked for without a device, follows from it; the GB300 has 152.)
constexpr int64_t kDispatchChunks = 152;
int chunk_of(int64_t T, int top_k) {
    return (int)std::min<int64_t>(kDispatchPairs / top_k, std::max<int64_t>(1, T / kDispatchChunks));
}
// no fewer than any number of tokens up to T has chunks
size_t chunks_bound(int64_t T, int top_k) {
    const int64_t most = kDispatchPairs / top_k;
    return (size_t)std::max((T + most - 1) / most, std::min<int64_t>(T, 2 * kDispatchChunks));
}

struct MoeWs {
    size_t pos, tiles, n_tiles, hist, xq, xs, hq, hs, o, total;
};
MoeWs moe_ws(int64_t T, int top_k, int64_t E, int64_t H, int64_t I) {
    const size_t P = (size_t)T * (size_t)top_k;
    MoeWs w;
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t at = off; off += up256(bytes); return at; };
    w.n_tiles = take(4);
    w.pos = take(P * 4);
    w.tiles = take((P / kSimtTileRows + std::min<size_t>(P, (size_t)E) + 1) * sizeof(Tile));
    w.hist = take((chunks_bound(T, top_k) + 1) * (size_t)E * 4);
    w.xq = take(P * (size_t)pad16(H));
    w.xs = take(P * (size_t)blocks_of(H) * 4);
    w.hq = take(P * (size_t)pad16(I));
    w.hs = take(P * (size_t)blocks_of(I) * 4);
    w.o = take(P * (size_t)std::max(pad4(H), I) * 4);   // the pairs' outputs (generic kernels: h before it)
    w.total = off;
    return w;
}

// The experts' two products, but for their operands.
struct MoeProducts {
    BlockGemm gate_up, down;
};
MoeProducts moe_products(int64_t T, int top_k, int64_t E, int64_t H, int64_t I, int tile_rows) {
    const int64_t pairs = T * top_k;
    BlockGemm g;
    std::memset(&g, 0, sizeof g);
    g.T = pairs;
    g.tile_rows = tile_rows;
    g.max_tiles = (int)std::min<int64_t>(pairs, pairs / tile_rows + std::min<int64_t>(E, pairs));
    g.expected_tiles = (int)std::min<int64_t>(g.max_tiles, pairs / tile_rows / 2 + std::min<int64_t>(E, pairs));
    g.groups = (int)E;
    MoeProducts p = {g, g};
    BlockGemm &gu = p.gate_up, &dn = p.down;
    gu.N = I; gu.K = H; gu.kb = (int)blocks_of(H);
    gu.w_group_rows = 2 * I; gu.up_rows = I;
    gu.up_scales = blocks_of(I) * blocks_of(H); gu.ws_group = 2 * gu.up_scales;
    gu.epi = BLOCK_SWIGLU;
    gu.ldo = I;
    gu.ldh = pad16(I);
    gu.hb = (int)blocks_of(I);
    dn.N = H; dn.K = I; dn.kb = gu.hb;
    dn.w_group_rows = H;
    dn.ws_group = blocks_of(H) * blocks_of(I);
    dn.epi = BLOCK_F32;
    dn.ldo = pad4(H);
    return p;
}
// a token or a few: gate_up finds its tiles in the ids, and its weights are requested while the tokens are dispatched
bool tiles_from_ids(int64_t pairs) { return pairs <= 32; }

bool moe_sizes_ok(int64_t T, int top_k, int64_t E, int64_t H, int64_t I) {
    return T > 0 && top_k > 0 && E > 0 && H > 0 && I > 0 && top_k <= MSE_ROUTE_MAX_TOP_K &&
           E <= MSE_ROUTE_MAX_EXPERTS && T * top_k <= kMaxRows && T <= kMaxRows && H <= kMaxInner && I <= kMaxInner;
}

// weight rows are 32-bit coordinates
bool moe_coordinates_ok(int64_t E, int64_t H, int64_t I) { return E * 2 * I <= kMaxRows && E * H <= kMaxRows; }

}  // namespace

extern "C" {

mse_status moe_route(const void *logits, mse_dtype logits_dtype, int64_t T, int64_t E, int64_t ld, const float *bias,
                     mse_score scoring, int n_group, int topk_group, int group_top, int top_k, int renormalise,
                     float scale, int32_t *ids, float *weights, int64_t capacity, void *stream) {
    if (!logits || !ids || !weights || T <= 0 || E <= 0 || ld < E || E > MSE_ROUTE_MAX_EXPERTS || T > kMaxRows ||
        ld > kMaxPitch ||
        (logits_dtype != MSE_BF16 && logits_dtype != MSE_F32) ||
        (scoring != MSE_SCORE_SOFTMAX && scoring != MSE_SCORE_SIGMOID) || n_group <= 0 ||
        n_group > MSE_ROUTE_MAX_GROUPS || topk_group <= 0 || topk_group > n_group ||
        (group_top != 1 && group_top != 2) || top_k <= 0 || top_k > MSE_ROUTE_MAX_TOP_K)
        return MSE_ERR_INVALID_ARG;
    if (E % n_group != 0) return MSE_ERR_NOT_DIVISIBLE;
    if (top_k > topk_group * (E / n_group)) return MSE_ERR_INVALID_ARG;
    if (capacity < T * top_k) return MSE_ERR_GEOMETRY;
    DeviceView d;
    const mse_status st = device_view(&d);
    if (st != MSE_OK) return st;
    begin_untracked_call(stream);
    RouteParams p;
    p.logits = logits; p.bf16_logits = logits_dtype == MSE_BF16;
    p.T = T; p.ld = ld; p.E = (int)E; p.bias = bias;
    p.sigmoid = scoring == MSE_SCORE_SIGMOID;
    // where every group stays there are none to choose
    p.n_group = topk_group == n_group ? 1 : n_group;
    p.group_size = (int)(E / p.n_group); p.topk_group = topk_group; p.group_top = group_top;
    p.top_k = top_k; p.renormalise = renormalise != 0; p.scale = scale;
    p.ids = ids; p.weights = weights;
    return from_cuda(launch_route(p, d.sm_count, pdl_enabled(), static_cast<cudaStream_t>(stream)));
}

mse_status fp8_block_quantise(const mse_bf16 *x, int64_t rows, int64_t K, int64_t ldx, int block_rows, uint8_t *q,
                              int64_t ldq, int64_t q_capacity, float *scales, int64_t scales_capacity, void *stream) {
    if (!x || !q || !scales || rows <= 0 || K <= 0 || ldx < K || ldq < K || (block_rows != 1 && block_rows != kBlock) ||
        rows > kMaxRows || K > kMaxInner || ldx > kMaxPitch || ldq > kMaxPitch)
        return MSE_ERR_INVALID_ARG;
    const int64_t scale_rows = block_rows == 1 ? rows : blocks_of(rows);
    if (block_rows != 1 && scale_rows * blocks_of(K) > INT32_MAX) return MSE_ERR_INVALID_ARG;   // a CTA for each block
    if (q_capacity < (rows - 1) * ldq + K || scales_capacity < scale_rows * blocks_of(K)) return MSE_ERR_GEOMETRY;
    DeviceView d;
    const mse_status st = device_view(&d);
    if (st != MSE_OK) return st;
    begin_untracked_call(stream);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (block_rows == 1)
        return from_cuda(launch_quantise_rows(x, rows, K, ldx, q, ldq, scales, d.sm_count, pdl_enabled(), s));
    return from_cuda(launch_quantise_tiles(x, rows, K, ldx, q, ldq, scales, pdl_enabled(), s));
}

mse_status fp8_block_matmul(const uint8_t *xq, int64_t ldx, const float *xs, const uint8_t *wq, int64_t ldw,
                            const float *ws, int64_t T, int64_t N, int64_t K, void *out, mse_dtype out_dtype,
                            int64_t out_capacity, void *stream) {
    mse_status st = check_matmul(xq, ldx, xs, wq, ldw, ws, T, N, K, out, out_dtype, out_capacity);
    if (st != MSE_OK) return st;
    DeviceView d;
    if ((st = device_view(&d)) != MSE_OK) return st;
    bool tensorcore = false;
    if ((st = choose_tensorcore(tc_operands(xq, ldx, wq, ldw), &tensorcore)) != MSE_OK) return st;
    begin_untracked_call(stream);
    return run_product(plain_product(xq, ldx, xs, wq, ldw, ws, T, N, K, out, out_dtype, d.sm_count), tensorcore, d,
                       static_cast<cudaStream_t>(stream));
}

size_t fp8_block_linear_workspace_bytes(int64_t T, int64_t N, int64_t K) {
    if (T <= 0 || N <= 0 || K <= 0 || T > kMaxRows || N > kMaxInner || K > kMaxInner) return 0;
    return linear_ws(T, K).total;
}

mse_status fp8_block_linear(const mse_bf16 *x, int64_t ldx, const uint8_t *wq, int64_t ldw, const float *ws, int64_t T,
                            int64_t N, int64_t K, void *y, mse_dtype y_dtype, int64_t y_capacity, void *workspace,
                            size_t workspace_bytes, void *stream) {
    mse_status st = check_matmul(x, ldx, x, wq, ldw, ws, T, N, K, y, y_dtype, y_capacity);
    if (st != MSE_OK) return st;
    const LinearWs L = linear_ws(T, K);
    if (!workspace || workspace_bytes < L.total || !aligned256(workspace)) return MSE_ERR_WORKSPACE;
    DeviceView d;
    if ((st = device_view(&d)) != MSE_OK) return st;
    uint8_t *xq = static_cast<uint8_t *>(workspace) + L.q_off;
    float *xs = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + L.s_off);
    const int64_t ldq = pad16(K);
    bool tensorcore = false;
    if ((st = choose_tensorcore(tc_operands(xq, ldq, wq, ldw), &tensorcore)) != MSE_OK) return st;
    begin_untracked_call(stream);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    BlockGemm g = plain_product(xq, ldq, xs, wq, ldw, ws, T, N, K, y, y_dtype, d.sm_count);
    // (y over x: the product's CTAs would write y while others still round x)
    const bool apart = disjoint(x, ((T - 1) * ldx + K) * 2, y, T * N * (y_dtype == MSE_F32 ? 4 : 2));
    if (tensorcore && apart && rounds_itself(T, N, K)) {
        g.x = x;
        g.ldxb = ldx;
        g.x_wide = ldx % 8 == 0 && aligned16(x);
        return run_product(g, tensorcore, d, s);
    }
    if ((st = from_cuda(launch_quantise_rows(x, T, K, ldx, xq, ldq, xs, d.sm_count, pdl_enabled(), s))) != MSE_OK)
        return st;
    g.weights_early = 1;
    return run_product(g, tensorcore, d, s);
}

size_t moe_experts_workspace_bytes(int64_t T, int top_k, int64_t E, int64_t H, int64_t I) {
    return moe_sizes_ok(T, top_k, E, H, I) ? moe_ws(T, top_k, E, H, I).total : 0;
}

mse_status moe_experts_forward(const mse_bf16 *x, int64_t T, int64_t H, const int32_t *ids, const float *weights,
                               int top_k, const uint8_t *w_gate_up, int64_t ld_gate_up, const float *s_gate_up,
                               const uint8_t *w_down, int64_t ld_down, const float *s_down, int64_t E, int64_t I,
                               int64_t first_expert, const mse_bf16 *shared, mse_bf16 *y, int64_t y_capacity,
                               void *workspace, size_t workspace_bytes, void *stream) {
    if (!x || !ids || !weights || !w_gate_up || !s_gate_up || !w_down || !s_down || !y ||
        !moe_sizes_ok(T, top_k, E, H, I) || ld_gate_up < H || ld_down < I || ld_gate_up > kMaxPitch ||
        ld_down > kMaxPitch || first_expert < 0)
        return MSE_ERR_INVALID_ARG;
    if (y_capacity < T * H) return MSE_ERR_GEOMETRY;
    const MoeWs L = moe_ws(T, top_k, E, H, I);
    if (!workspace || workspace_bytes < L.total || !aligned256(workspace)) return MSE_ERR_WORKSPACE;
    DeviceView d;
    mse_status st = device_view(&d);
    if (st != MSE_OK) return st;
    bool tensorcore = false;
    const bool tc_ok = aligned16(w_gate_up) && aligned16(w_down) && ld_gate_up % 16 == 0 && ld_down % 16 == 0 &&
                       moe_coordinates_ok(E, H, I);
    if ((st = choose_tensorcore(tc_ok, &tensorcore)) != MSE_OK) return st;
    begin_untracked_call(stream);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool pdl = pdl_enabled();
    uint8_t *w = static_cast<uint8_t *>(workspace);
    const int64_t pairs = T * top_k;

    DispatchParams dp;
    std::memset(&dp, 0, sizeof dp);
    dp.x = x; dp.T = T; dp.H = H; dp.align = align_of(x, H); dp.ids = ids; dp.top_k = top_k; dp.first_expert = first_expert; dp.E = (int)E;
    dp.chunk = chunk_of(T, top_k);
    if (pairs > kCountAllPairs) dp.hist = reinterpret_cast<int *>(w + L.hist);   // the ids are counted once, by two kernels of their own
    dp.n_chunks = (int)((T + dp.chunk - 1) / dp.chunk);
    // the k-blocks of a chunk over several CTAs, up to eight per SM (the rows are written by many warps at once: 4096 tokens of
    // 7168 x 8 in 60 us, 230 on 128 CTAs)
    dp.splits = (int)std::max<int64_t>(1, std::min<int64_t>(blocks_of(H) / 4, 8 * d.sm_count / dp.n_chunks));
    dp.pos = reinterpret_cast<int32_t *>(w + L.pos);
    dp.tiles = reinterpret_cast<Tile *>(w + L.tiles);
    dp.n_tiles = reinterpret_cast<int *>(w + L.n_tiles);
    dp.tile_rows = tensorcore ? expert_tile_rows(pairs / E) : kSimtTileRows;
    dp.xq = w + L.xq; dp.ldq = pad16(H);
    dp.xs = reinterpret_cast<float *>(w + L.xs);
    if ((st = from_cuda(launch_dispatch(dp, pdl, s))) != MSE_OK) return st;

    float *o = reinterpret_cast<float *>(w + L.o);
    MoeProducts p = moe_products(T, top_k, E, H, I, dp.tile_rows);
    BlockGemm &gu = p.gate_up, &dn = p.down;
    gu.tiles = dn.tiles = dp.tiles;
    gu.n_tiles = dn.n_tiles = dp.n_tiles;
    gu.xq = dp.xq; gu.ldx = dp.ldq; gu.xs = dp.xs;
    gu.wq = w_gate_up; gu.ldw = ld_gate_up; gu.ws = s_gate_up;
    gu.out = o;
    gu.hq = w + L.hq;
    gu.hs = reinterpret_cast<float *>(w + L.hs);
    if (tensorcore && tiles_from_ids(pairs) && pdl) {
        gu.ids = ids;
        gu.pairs = (int)pairs;
        gu.first_expert = first_expert;
        gu.weights_early = 1;
    }
    if ((st = run_product(gu, tensorcore, d, s)) != MSE_OK) return st;
    if (!tensorcore && (st = from_cuda(launch_quantise_f32(o, dp.n_tiles, dp.tiles, gu.max_tiles, I, gu.hq, gu.ldh, gu.hs, pdl, s))) !=
        MSE_OK)
        return st;
    dn.xq = gu.hq; dn.ldx = gu.ldh; dn.xs = gu.hs;
    dn.wq = w_down; dn.ldw = ld_down; dn.ws = s_down;
    dn.out = o;
    dn.weights_early = 1;   // (and the tiles: the gate_up launch lets this one start after its own wait; the CTA-pair kernel
                            // waits for all of it)
    if ((st = run_product(dn, tensorcore, d, s)) != MSE_OK) return st;
    return from_cuda(launch_combine(o, dn.ldo, dp.pos, weights, top_k, shared, y, T, H, d.sm_count, pdl, s));
}

mse_status mse_fp8_launch_plan(int64_t T, int64_t N, int64_t K, int32_t *out) {
    if (!out || T <= 0 || N <= 0 || K <= 0 || T > kMaxRows || N > kMaxInner || K > kMaxInner) return MSE_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i) out[i] = 0;
    DeviceView d;
    mse_status st = device_view(&d);
    if (st != MSE_OK) return st;
    bool tensorcore = false;
    if ((st = choose_tensorcore(true, &tensorcore)) != MSE_OK || !tensorcore) return st;
    const BlockGemm g = plain_product(nullptr, pad16(K), nullptr, nullptr, pad16(K), nullptr, T, N, K, nullptr, MSE_BF16, d.sm_count);
    const Split split = g.tile_rows == 256 ? pair_split(g, d.sm_count) : cols_split(g, d.sm_count);
    out[0] = g.tile_rows;
    out[1] = split.parts;
    out[2] = (int32_t)std::min<int64_t>(split.ctas, INT32_MAX);
    out[3] = rounds_itself(T, N, K);
    return MSE_OK;
}

mse_status mse_moe_launch_plan(int64_t T, int top_k, int64_t E, int64_t H, int64_t I, int32_t *out) {
    if (!out || !moe_sizes_ok(T, top_k, E, H, I)) return MSE_ERR_INVALID_ARG;
    for (int i = 0; i < 8; ++i) out[i] = 0;
    DeviceView d;
    mse_status st = device_view(&d);
    if (st != MSE_OK) return st;
    bool tensorcore = false;
    if ((st = choose_tensorcore(moe_coordinates_ok(E, H, I), &tensorcore)) != MSE_OK) return st;
    out[6] = T * top_k > kCountAllPairs;
    if (!tensorcore) return MSE_OK;
    const MoeProducts p = moe_products(T, top_k, E, H, I, expert_tile_rows(T * top_k / E));
    BlockGemm g[2] = {p.gate_up, p.down};
    static const Tile some = {};   // a grouped product; its tiles are the call's
    out[0] = g[0].tile_rows;
    for (int i = 0; i < 2; ++i) {
        g[i].tiles = &some;
        const Split split = out[0] == 256 ? pair_split(g[i], d.sm_count) : cols_split(g[i], d.sm_count);
        out[1 + 2 * i] = split.parts;
        out[2 + 2 * i] = (int32_t)std::min<int64_t>(split.ctas, INT32_MAX);
    }
    out[5] = tiles_from_ids(T * top_k) && pdl_enabled();
    return MSE_OK;
}

}  // extern "C"
