// C-ABI entry points of the sorted rows and of the products in 8-bit integers: argument validation (before any CUDA
// call), workspace carving and kernel choice.
#include <algorithm>
#include <cstring>
#include <initializer_list>

#include "device.h"
#include "sorted.h"

using namespace mse;
using namespace mse::sorted;

namespace {

size_t up256(size_t v) { return (v + 255) / 256 * 256; }
bool aligned256(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
// Memory of an argument, and whether what a call writes lies apart from what it reads and from what else it writes: CTAs read while
// others write.  (Of a null pointer there is none.)
struct Range {
    uintptr_t from, to;
};
Range range(const void *p, int64_t bytes) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    return {at, p ? at + (uintptr_t)bytes : at};
}
bool apart(std::initializer_list<Range> written, std::initializer_list<Range> read) {
    for (const Range *w = written.begin(); w != written.end(); ++w) {
        auto meets = [w](const Range &o) { return w->from < o.to && o.from < w->to; };
        if (std::any_of(read.begin(), read.end(), meets) || std::any_of(written.begin(), w, meets)) return false;
    }
    return true;
}
mse_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MSE_OK : MSE_ERR_CUDA; }
bool dtype_ok(mse_dtype d) { return d == MSE_BF16 || d == MSE_F32; }
int64_t size_of(mse_dtype d) { return d == MSE_F32 ? 4 : 2; }
// bytes from the first to the last value of rows with a pitch
int64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t size) { return ((rows - 1) * ld + cols) * size; }

// ------------------------------------------------------------------ sort
// Up to this many pairs every CTA counts all ids itself.
constexpr int64_t kCountAllPairs = 4096;
// Tokens of a chunk: about as many chunks as the GB300 has SMs, as far as a chunk's pairs reach.  (A constant, because the
// workspace's size, asked for without a device, follows from it.)
constexpr int64_t kChunks = 152;
int chunk_of(int64_t T, int top_k) {
    return (int)std::min<int64_t>(kSortThreads / top_k, std::max<int64_t>(1, T / kChunks));
}
// no fewer than any number of tokens up to T has chunks
size_t chunks_bound(int64_t T, int top_k) {
    const int64_t most = kSortThreads / top_k;
    return (size_t)std::max((T + most - 1) / most, std::min<int64_t>(T, 2 * kChunks));
}
bool sort_sizes_ok(int64_t T, int top_k, int64_t E) {
    return T > 0 && top_k > 0 && E > 0 && top_k <= MSE_ROUTE_MAX_TOP_K && E <= MSE_ROUTE_MAX_EXPERTS && T <= kMaxRows &&
           T * top_k <= kMaxRows;
}
size_t sort_ws(int64_t T, int top_k, int64_t E) {
    return up256(T * top_k > kCountAllPairs ? (chunks_bound(T, top_k) + 1) * (size_t)E * 4 : 4);
}

// ------------------------------------------------------------------ 8-bit integers
// tokens as the product's kernels take them, and their scales
struct Int8Ws {
    size_t q_off, s_off, total;
};
Int8Ws int8_ws(int64_t T, int64_t K) {
    Int8Ws w;
    w.q_off = 0;
    w.s_off = up256((size_t)T * (size_t)((K + 63) / 64 * 64) * 2);
    w.total = w.s_off + up256((size_t)T * 4);
    return w;
}
bool int8_sizes_ok(int64_t T, int64_t N, int64_t K, int64_t groups) {
    return T > 0 && N > 0 && K > 0 && groups > 0 && T <= kMaxRows && N <= kMaxInner && K <= kMaxInt8Inner &&
           groups <= MSE_ROUTE_MAX_EXPERTS;
}

mse_status check_product(const void *x, int64_t ldx, const void *xs, const void *wq, int64_t ldw, const void *ws, int64_t T,
                         int64_t N, int64_t K, int64_t groups, const void *out, mse_dtype dtype, int64_t capacity,
                         const void *workspace, size_t bytes) {
    if (!x || !xs || !wq || !ws || !out || !int8_sizes_ok(T, N, K, groups) || ldx < K || ldw < K || ldx > kMaxPitch ||
        ldw > kMaxPitch || !dtype_ok(dtype) || groups * N > kMaxRows)
        return MSE_ERR_INVALID_ARG;
    if (capacity < T * N) return MSE_ERR_GEOMETRY;
    if (!workspace || bytes < int8_ws(T, K).total || !aligned256(workspace)) return MSE_ERR_WORKSPACE;
    return MSE_OK;
}

// What a product reads and writes: of int8_linear, whose xs are in the workspace, x in place of xq.
struct ProductMemory {
    Range x, xs, wq, ws, offsets, out, space;
};
ProductMemory memory_of(const Int8Gemm &g, const void *x, int64_t ldx, int64_t x_size, const void *workspace) {
    const int64_t channels = g.groups * g.N;
    return {range(x, span(g.T, g.K, ldx, x_size)), range(g.xs, g.T * 4), range(g.wq, span(channels, g.K, g.ldw, 1)),
            range(g.ws, channels * 4), range(g.offsets, (g.groups + 1) * (int64_t)4), range(g.out, g.T * g.N * (g.out_f32 ? 4 : 2)),
            range(workspace, (int64_t)int8_ws(g.T, g.K).total)};
}
// (every part of a row of out takes all of a row of x)
bool out_apart(const ProductMemory &m, bool over_x) {
    return apart({m.out}, {over_x ? range(nullptr, 0) : m.x, m.xs, m.wq, m.ws, m.offsets, m.space});
}
bool space_apart(const ProductMemory &m) { return apart({m.space}, {m.x, m.xs, m.wq, m.ws, m.offsets}); }
int64_t pitch16(int64_t K) { return (K + 63) / 64 * 64; }   // of tokens in fp16

// Token rows of a tile: up to 4 the kernel for few, 16 to 64 the swap-AB kernel, 256 the CTA-pair kernel.
//
// A plain product by its rows.  (us with the kernel for few, of int8 rows, and the swap-AB kernel: 2 x 2112 x 7168 5.6, 9.8; 4 x
// 2112 x 7168 7.4, 9.9; 4 x 12288 x 7168 20.2, 20.5; 8 x 2112 x 7168 10.7, 9.9; 8 x 12288 x 7168 28, 20.6.)  Grouped rows by those
// expected of a group, but for a token's or two's rows, of which few groups have more than two.  (us with tiles of 2, 4 and 16, 8
// experts a token: 1 token of 32 x 4096 x 7168 40.8, 46.1, 43.4, of 32 x 7168 x 2048 22.2, 22.5, 27.7; 2 tokens of 32 x 4096 x
// 7168 69, 70, 76; 4 tokens 113, 119, 104; 16 tokens of 32 of 128 experts 233, 181, 94.)  The rule does not look at the groups:
// where few have these rows, tiles of 2 read a group's weights again for every two rows (8 rows of 4096 x 7168 with tiles of 2 and
// 16: in 8 groups 39.8, 41.8, in 4 31.6, 25.0, in one 21.4, 13.5; 16 rows in one 33.4, 14.4).
//
// More rows take tiles of 64 on the swap-AB kernel or the CTA pairs, whichever a model expects to be done first, in units of 10 ns:
// two swap-AB CTAs on an SM take 0.6 us for a k-block each and 4 us for a tile besides, 2.5 more where its k-blocks are split; a CTA
// pair 0.75 us for a k-block and 5 us in all, 3 more where two share a tile's.  us with tiles of 64 and of 256, * where the rule
// takes the slower:
//
//   rows x 12288 x 7168     65 37.6 40.4   160 38.2 46.6   200 62.5 47.2   256 63.5 47.3   320 69.7 83.6*  384 70.9 84.1*
//                          512 100 86.9    768 135 88.5   1024 186 128
//   rows x 2112 x 7168     128 14.8 25.1   256 16.9 30.2   384 24.2 30.7   512 24.7 31.0   768 36.6 32.1  1024 37.5 33.2
//   rows x 7168 x 2048     128 13.1 15.6   320 15.6 17.7   512 25.5 18.1   768 37.0 29.0  1024 41.0 29.7
//   rows x 4096 x 2048     128 10.8 14.6   400 15.1 17.2   800 24.9 18.1
//   rows of each of 32 experts of 4096 x 2048   32 63.4 83.5*   64 65.8 85.5*   96 105 87.1   128 110 88.5   256 200 107
//   rows of each of 8 experts of 4096 x 7168    32 46.4 77.3    64 49.3 78.2*  128 81.0 82.4*  256 149 98.7
//
// What the model has wrong: a tile of up to 128 tokens counts as half of one, though loads and conversions take nearly as long as a whole
// one's, and two of them as one pair's turn.  (Tiles of 128 on the swap-AB kernel were never the fastest by more than a few per cent.)
// A rank that holds a part of the experts is judged by all rows of xq, its own or not: 128 tokens to 8 of 128 experts of 4096 x 2048,
// 32 of them here, 298 rows, take 81.4 as 1024 rows and 55.7 passed as 298; 256 tokens 82.6 and 61.6.
constexpr int64_t kFewRows = 4, kFewGroupedRows = 16;
int tile_rows_of(const Int8Gemm &g, int sm_count) {
    const int few = g.offsets ? (g.T <= kFewGroupedRows ? 2 : 0) : g.T <= kFewRows ? (g.T > 2 ? 4 : (int)g.T) : 0;
    if (few > 0 && int8_few_serves(few, g.K)) return few;
    const int64_t rows = g.T / g.groups;
    if (rows <= (g.offsets ? 8 : 16)) return 16;
    if (rows <= (g.offsets ? 24 : 32)) return 32;
    // a group's last tile is half full on the average; a pair's tile of up to 128 rows counts half
    const int64_t kb = (g.K + 127) / 128, part = g.offsets ? g.groups / 2 : 0;
    const int64_t cols = ((g.T + 63) / 64 + part) * ((g.N + 127) / 128), halves = ((g.T + 127) / 128 + part) * ((g.N + 255) / 256);
    const int64_t cp = int8_cols_parts(cols, (int)kb, sm_count), pp = int8_pair_parts(int8_pair_tiles(g), (int)kb);
    const int64_t waves = (cols * cp + 2 * sm_count - 1) / (2 * sm_count);
    const int64_t rounds = ((halves + 1) / 2 * pp + sm_count / 2 - 1) / (sm_count / 2);
    const int64_t cols_time = waves * (kb * 60 / cp + 400 + (cp > 1 ? 250 : 0));
    const int64_t pair_time = rounds * kb * 75 / pp + 500 + (pp > 1 ? 300 : 0);
    // (a swap-AB grid has at most 65,535 token tiles)
    return pair_time < cols_time || int8_cols_slots(g, 64) > 65535 ? 256 : 64;
}

// One launch, whose kernel rounds the token itself: every CTA rounds it.  (us with one launch and two: 1 x 2112 x 7168 6.3, 7.6; two
// tokens 8.3, 8.1.)
bool rounds_itself(int tile_rows) { return tile_rows == 1; }

bool tensorcore_ok(const Int8Gemm &g) { return (reinterpret_cast<uintptr_t>(g.wq) & 15u) == 0 && g.ldw % 16 == 0; }

mse_status run_tensorcore(const Int8Gemm &g, int tile_rows, const DeviceView &d, cudaStream_t s) {
    if (tile_rows == 256) return launch_int8_pair(g, d.sm_count, pdl_enabled(), s);
    return launch_int8_cols(g, tile_rows, d.sm_count, pdl_enabled(), s);
}

// int8 rows: expanded to fp16 in the workspace for the tensor cores
mse_status run_product(Int8Gemm g, const DeviceView &d, void *workspace, cudaStream_t s) {
    g.wait_limit_ns = wait_limit_ns();
    g.err = d.err;
    bool fast = false;
    mse_status st = choose_tensorcore(tensorcore_ok(g), &fast);
    if (st != MSE_OK) return st;
    if (!fast) return from_cuda(launch_int8_simt(g, pdl_enabled(), s));
    const int tile_rows = tile_rows_of(g, d.sm_count);
    if (tile_rows <= 4) return from_cuda(launch_int8_few(g, tile_rows, nullptr, 0, 0, false, d.sm_count, pdl_enabled(), s));
    g.ldx16 = pitch16(g.K);
    uint16_t *x16 = static_cast<uint16_t *>(workspace);
    st = from_cuda(launch_int8_expand(g.xq, g.ldx, g.T, g.K, g.offsets ? g.offsets + g.groups : nullptr, x16, g.ldx16, d.sm_count,
                                      pdl_enabled(), s));
    if (st != MSE_OK) return st;
    g.x16 = x16;
    return run_tensorcore(g, tile_rows, d, s);
}

Int8Gemm product(const int8_t *xq, int64_t ldx, const float *xs, const int32_t *offsets, int64_t groups, const int8_t *wq,
                 int64_t ldw, const float *ws, int64_t T, int64_t N, int64_t K, void *out, mse_dtype dtype) {
    Int8Gemm g;
    std::memset(&g, 0, sizeof g);
    g.T = T;
    g.xq = xq; g.ldx = ldx; g.xs = xs;
    g.offsets = offsets; g.groups = (int)groups;
    g.wq = wq; g.ldw = ldw; g.ws = ws;
    g.N = N; g.K = K;
    g.out = out; g.out_f32 = dtype == MSE_F32;
    return g;
}

}  // namespace

extern "C" {

size_t moe_sort_workspace_bytes(int64_t T, int top_k, int64_t E) { return sort_sizes_ok(T, top_k, E) ? sort_ws(T, top_k, E) : 0; }

mse_status moe_sort(const void *x, int value_bytes, int64_t T, int64_t H, int64_t ldx, const int32_t *ids, int top_k, int64_t E,
                    int64_t first_expert, const float *scales, void *rows, int64_t ldr, int64_t rows_capacity,
                    float *row_scales, int32_t *place, int32_t *offsets, void *workspace, size_t workspace_bytes, void *stream) {
    if (!x || !ids || !rows || !place || !offsets || (scales != nullptr) != (row_scales != nullptr) ||
        (value_bytes != 1 && value_bytes != 2 && value_bytes != 4) || !sort_sizes_ok(T, top_k, E) || H <= 0 || H > kMaxInner ||
        ldx < H || ldr < H || ldx > kMaxPitch || ldr > kMaxPitch || first_expert < 0)
        return MSE_ERR_INVALID_ARG;
    const int64_t pairs = T * top_k;
    if (rows_capacity < (pairs - 1) * ldr + H) return MSE_ERR_GEOMETRY;
    const Range x_range = range(x, span(T, H, ldx, value_bytes)), ids_range = range(ids, pairs * 4), scales_range = range(scales, T * 4),
                offsets_range = range(offsets, (E + 1) * 4), space = range(workspace, (int64_t)sort_ws(T, top_k, E));
    if (!apart({range(rows, span(pairs, H, ldr, value_bytes)), range(place, pairs * 4), range(row_scales, pairs * 4)},
               {x_range, ids_range, scales_range, offsets_range, space}))
        return MSE_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < sort_ws(T, top_k, E) || !aligned256(workspace)) return MSE_ERR_WORKSPACE;
    DeviceView d;
    const mse_status st = device_view(&d);
    if (st != MSE_OK) return st;
    // (Only with a device: callers that check arguments without one give several of them one address.)
    if (!apart({offsets_range, space}, {x_range, ids_range, scales_range})) return MSE_ERR_INVALID_ARG;
    begin_untracked_call(stream);
    SortParams p;
    std::memset(&p, 0, sizeof p);
    p.x = static_cast<const uint8_t *>(x); p.T = T; p.row_bytes = H * value_bytes; p.ldx = ldx * value_bytes;
    p.ids = ids; p.top_k = top_k; p.first_expert = first_expert; p.E = (int)E;
    p.scales = scales;
    p.rows = static_cast<uint8_t *>(rows); p.ldr = ldr * value_bytes;
    p.row_scales = row_scales;
    p.place = place; p.offsets = offsets;
    p.chunk = chunk_of(T, top_k);
    p.n_chunks = (int)((T + p.chunk - 1) / p.chunk);
    if (pairs > kCountAllPairs) p.hist = static_cast<int *>(workspace);
    const uint64_t bits = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(rows) | (uint64_t)p.ldx |
                          (uint64_t)p.ldr | (uint64_t)p.row_bytes | 16u;
    p.unit = (int)(bits & (~bits + 1));
    // the copies of a chunk over several CTAs, of 1 KB for each warp at least (of half as much where there are few: one token of 7168 in
    // bf16 to eight experts 3.6 us, 4.3) and, beyond eight CTAs an SM, of 4 KB
    p.few = T * p.row_bytes <= 65536;
    const int64_t bytes = p.row_bytes * p.chunk, room = 16 * d.sm_count / p.n_chunks, least = p.few ? 4096 : 8192;
    p.splits = (int)std::max<int64_t>(1, std::min(std::max(std::min((bytes + least - 1) / least, room / 2), bytes / 32768), room));
    return from_cuda(launch_sort(p, pdl_enabled(), static_cast<cudaStream_t>(stream)));
}

mse_status moe_unsort(const void *rows, mse_dtype rows_dtype, int64_t n_rows, int64_t ldr, const int32_t *place,
                      const float *weights, int64_t T, int64_t H, int top_k, const void *base, void *y, mse_dtype y_dtype,
                      int64_t y_capacity, void *stream) {
    if (!rows || !place || !y || !dtype_ok(rows_dtype) || !dtype_ok(y_dtype) || T <= 0 || H <= 0 || top_k <= 0 ||
        n_rows <= 0 || T > kMaxRows || n_rows > kMaxRows || H > kMaxInner || top_k > MSE_ROUTE_MAX_TOP_K || ldr < H ||
        ldr > kMaxPitch)
        return MSE_ERR_INVALID_ARG;
    if (y_capacity < T * H) return MSE_ERR_GEOMETRY;
    const int64_t y_bytes = T * H * size_of(y_dtype), pairs_bytes = T * top_k * 4;
    if (!apart({range(y, y_bytes)}, {range(rows, span(n_rows, H, ldr, size_of(rows_dtype))), range(place, pairs_bytes),
                                     range(weights, pairs_bytes), range(base == y ? nullptr : base, y_bytes)}))
        return MSE_ERR_INVALID_ARG;
    DeviceView d;
    const mse_status st = device_view(&d);
    if (st != MSE_OK) return st;
    begin_untracked_call(stream);
    UnsortParams p;
    p.rows = rows; p.n_rows = n_rows; p.ldr = ldr;
    p.place = place; p.weights = weights; p.top_k = top_k;
    p.base = base; p.y = y; p.T = T; p.H = H;
    p.rows_f32 = rows_dtype == MSE_F32; p.y_f32 = y_dtype == MSE_F32;
    return from_cuda(launch_unsort(p, d.sm_count, pdl_enabled(), static_cast<cudaStream_t>(stream)));
}

mse_status moe_unsort_backward(const void *dy, mse_dtype dy_dtype, const int32_t *place, const float *weights,
                               const void *rows, mse_dtype rows_dtype, int64_t ldr, int64_t n_rows, int64_t T, int64_t H,
                               int top_k, void *drows, int64_t ldd, int64_t drows_capacity, float *dweights, void *stream) {
    if (!dy || !place || !drows || !dtype_ok(dy_dtype) || !dtype_ok(rows_dtype) || (weights != nullptr) != (dweights != nullptr) ||
        (weights && (!rows || ldr < H || ldr > kMaxPitch)) || T <= 0 || H <= 0 || top_k <= 0 || n_rows <= 0 || T > kMaxRows ||
        n_rows > kMaxRows || H > kMaxInner || top_k > MSE_ROUTE_MAX_TOP_K || ldd < H || ldd > kMaxPitch)
        return MSE_ERR_INVALID_ARG;
    if (drows_capacity < (n_rows - 1) * ldd + H) return MSE_ERR_GEOMETRY;
    const int64_t size = size_of(rows_dtype), pairs_bytes = T * top_k * 4;
    const Range dy_range = range(dy, T * H * size_of(dy_dtype)), place_range = range(place, pairs_bytes),
                rows_range = range(weights ? rows : nullptr, span(n_rows, H, ldr, size)), no_range = range(nullptr, 0);
    const bool in_place = rows == drows && ldr == ldd;
    if (!apart({range(drows, span(n_rows, H, ldd, size)), range(dweights, pairs_bytes)}, {}) ||
        !apart({range(drows, span(n_rows, H, ldd, size))},
               {dy_range, place_range, range(weights, pairs_bytes), in_place ? no_range : rows_range}))
        return MSE_ERR_INVALID_ARG;
    DeviceView d;
    const mse_status st = device_view(&d);
    if (st != MSE_OK) return st;
    if (!apart({range(dweights, pairs_bytes)},   // (only with a device, as in moe_sort)
               {dy_range, place_range, rows_range, dweights == weights ? no_range : range(weights, pairs_bytes)}))
        return MSE_ERR_INVALID_ARG;
    begin_untracked_call(stream);
    UnsortBackwardParams p;
    p.dy = dy; p.place = place; p.weights = weights;
    p.rows = weights ? rows : nullptr; p.ldr = weights ? ldr : ldd;
    p.top_k = top_k;
    p.drows = drows; p.ldd = ldd; p.n_rows = n_rows;
    p.dweights = dweights;
    p.T = T; p.H = H;
    p.dy_f32 = dy_dtype == MSE_F32; p.rows_f32 = rows_dtype == MSE_F32;
    return from_cuda(launch_unsort_backward(p, d.sm_count, pdl_enabled(), static_cast<cudaStream_t>(stream)));
}

mse_status int8_quantise(const void *x, mse_dtype x_dtype, int64_t rows, int64_t K, int64_t ldx, int swiglu,
                         const int32_t *last, int8_t *q, int64_t ldq, int64_t q_capacity, float *scales, void *stream) {
    const int64_t width = swiglu ? 2 * K : K;
    if (!x || !q || !scales || !dtype_ok(x_dtype) || rows <= 0 || K <= 0 || rows > kMaxRows || K > kMaxInner || ldx < width ||
        ldq < K || ldx > kMaxPitch || ldq > kMaxPitch)
        return MSE_ERR_INVALID_ARG;
    if (q_capacity < (rows - 1) * ldq + K) return MSE_ERR_GEOMETRY;
    const Range x_range = range(x, span(rows, width, ldx, size_of(x_dtype))), last_range = range(last, 4), scales_range = range(scales, rows * 4);
    if (!apart({range(q, span(rows, K, ldq, 1))}, {x_range, last_range, scales_range})) return MSE_ERR_INVALID_ARG;
    DeviceView d;
    const mse_status st = device_view(&d);
    if (st != MSE_OK) return st;
    if (!apart({scales_range}, {x_range, last_range})) return MSE_ERR_INVALID_ARG;   // (only with a device, as in moe_sort)
    begin_untracked_call(stream);
    RoundParams p;
    p.x = x; p.rows = rows; p.K = K; p.ldx = ldx;
    p.f32 = x_dtype == MSE_F32; p.swiglu = swiglu != 0;
    p.last = last;
    p.q = q; p.ldq = ldq; p.half_out = 0; p.scales = scales;
    return from_cuda(launch_int8_round(p, d.sm_count, pdl_enabled(), static_cast<cudaStream_t>(stream)));
}

mse_status mse_int8_launch_plan(int64_t T, int64_t N, int64_t K, int64_t groups, int32_t *out) {
    if (!out || !int8_sizes_ok(T, N, K, groups > 0 ? groups : 1) || groups < 0 || std::max<int64_t>(groups, 1) * N > kMaxRows)
        return MSE_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i) out[i] = 0;
    DeviceView d;
    mse_status st = device_view(&d);
    if (st != MSE_OK) return st;
    static const int32_t some = 0;   // a grouped product; its offsets are the call's
    const Int8Gemm g = product(nullptr, 0, nullptr, groups > 0 ? &some : nullptr, std::max<int64_t>(groups, 1), nullptr,
                               (K + 15) / 16 * 16, nullptr, T, N, K, nullptr, MSE_BF16);
    bool fast = false;
    if ((st = choose_tensorcore(tensorcore_ok(g), &fast)) != MSE_OK || !fast) return st;
    out[0] = tile_rows_of(g, d.sm_count);
    out[1] = out[0] <= 4 ? 1
             : out[0] == 256
                 ? int8_pair_parts(int8_pair_tiles(g), (int)((K + 127) / 128))
                 : int8_cols_parts(int8_cols_slots(g, out[0]) * ((N + 127) / 128), (int)((K + 127) / 128), d.sm_count);
    out[2] = groups == 0 && rounds_itself(out[0]);
    return MSE_OK;
}

size_t int8_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t groups) {
    return int8_sizes_ok(T, N, K, groups) ? int8_ws(T, K).total : 0;
}

mse_status int8_matmul(const int8_t *xq, int64_t ldx, const float *xs, const int8_t *wq, int64_t ldw, const float *ws, int64_t T,
                       int64_t N, int64_t K, void *out, mse_dtype out_dtype, int64_t out_capacity, void *workspace,
                       size_t workspace_bytes, void *stream) {
    mse_status st = check_product(xq, ldx, xs, wq, ldw, ws, T, N, K, 1, out, out_dtype, out_capacity, workspace, workspace_bytes);
    if (st != MSE_OK) return st;
    const Int8Gemm g = product(xq, ldx, xs, nullptr, 1, wq, ldw, ws, T, N, K, out, out_dtype);
    const ProductMemory m = memory_of(g, xq, ldx, 1, workspace);
    if (!out_apart(m, false)) return MSE_ERR_INVALID_ARG;
    DeviceView d;
    if ((st = device_view(&d)) != MSE_OK) return st;
    if (!space_apart(m)) return MSE_ERR_INVALID_ARG;   // (only with a device, as in moe_sort)
    begin_untracked_call(stream);
    return run_product(g, d, workspace, static_cast<cudaStream_t>(stream));
}

mse_status int8_grouped_matmul(const int8_t *xq, int64_t ldx, const float *xs, const int32_t *offsets, int64_t groups,
                               const int8_t *wq, int64_t ldw, const float *ws, int64_t T, int64_t N, int64_t K, void *out,
                               mse_dtype out_dtype, int64_t out_capacity, void *workspace, size_t workspace_bytes,
                               void *stream) {
    if (!offsets) return MSE_ERR_INVALID_ARG;
    mse_status st =
        check_product(xq, ldx, xs, wq, ldw, ws, T, N, K, groups, out, out_dtype, out_capacity, workspace, workspace_bytes);
    if (st != MSE_OK) return st;
    const Int8Gemm g = product(xq, ldx, xs, offsets, groups, wq, ldw, ws, T, N, K, out, out_dtype);
    const ProductMemory m = memory_of(g, xq, ldx, 1, workspace);
    if (!out_apart(m, false)) return MSE_ERR_INVALID_ARG;
    DeviceView d;
    if ((st = device_view(&d)) != MSE_OK) return st;
    if (!space_apart(m)) return MSE_ERR_INVALID_ARG;   // (only with a device, as in moe_sort)
    begin_untracked_call(stream);
    return run_product(g, d, workspace, static_cast<cudaStream_t>(stream));
}

mse_status int8_linear(const void *x, mse_dtype x_dtype, int64_t ldx, const int8_t *wq, int64_t ldw, const float *ws, int64_t T,
                       int64_t N, int64_t K, void *y, mse_dtype y_dtype, int64_t y_capacity, void *workspace,
                       size_t workspace_bytes, void *stream) {
    if (!dtype_ok(x_dtype)) return MSE_ERR_INVALID_ARG;
    mse_status st = check_product(x, ldx, ws, wq, ldw, ws, T, N, K, 1, y, y_dtype, y_capacity, workspace, workspace_bytes);
    if (st != MSE_OK) return st;
    Int8Gemm g = product(nullptr, 0, nullptr, nullptr, 1, wq, ldw, ws, T, N, K, y, y_dtype);
    const ProductMemory m = memory_of(g, x, ldx, size_of(x_dtype), workspace);
    if (!out_apart(m, true)) return MSE_ERR_INVALID_ARG;
    DeviceView d;
    if ((st = device_view(&d)) != MSE_OK) return st;
    if (!space_apart(m)) return MSE_ERR_INVALID_ARG;   // (only with a device, as in moe_sort)
    begin_untracked_call(stream);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    float *xs = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + int8_ws(T, K).s_off);
    g.xs = xs;
    g.wait_limit_ns = wait_limit_ns();
    g.err = d.err;
    bool fast = false;
    if ((st = choose_tensorcore(tensorcore_ok(g), &fast)) != MSE_OK) return st;
    const int tile_rows = fast ? tile_rows_of(g, d.sm_count) : 0;
    // (y over x: the product's CTAs would write y while others still round x)
    if (fast && rounds_itself(tile_rows) && apart({m.out}, {m.x}))
        return from_cuda(launch_int8_few(g, tile_rows, x, x_dtype == MSE_F32, ldx, false, d.sm_count, pdl_enabled(), s));
    RoundParams p;
    p.x = x; p.rows = T; p.K = K; p.ldx = ldx;
    p.f32 = x_dtype == MSE_F32; p.swiglu = 0;
    p.last = nullptr;
    p.q = workspace; p.ldq = pitch16(K); p.half_out = fast && tile_rows > 4; p.scales = xs;
    if ((st = from_cuda(launch_int8_round(p, d.sm_count, pdl_enabled(), s))) != MSE_OK) return st;
    g.xq = static_cast<const int8_t *>(workspace); g.ldx = p.ldq;
    if (!fast) return from_cuda(launch_int8_simt(g, pdl_enabled(), s));
    if (tile_rows <= 4) return from_cuda(launch_int8_few(g, tile_rows, nullptr, 0, 0, true, d.sm_count, pdl_enabled(), s));
    g.x16 = static_cast<const uint16_t *>(workspace); g.ldx16 = p.ldq;
    return run_tensorcore(g, tile_rows, d, s);
}

}  // extern "C"
