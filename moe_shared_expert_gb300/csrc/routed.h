// Internal interfaces of the routed-expert operators: routing, 8-bit block products, dispatch.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mse.h"

namespace mse {
namespace routed {

constexpr int kBlock = 128;              // rows or columns that share a scale
inline int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }
inline int64_t pad16(int64_t n) { return (n + 15) / 16 * 16; }
inline int64_t pad4(int64_t n) { return (n + 3) / 4 * 4; }

// ------------------------------------------------------------------ routing
struct RouteParams {
    const void *logits;
    int bf16_logits;
    int64_t T, ld;
    int E;
    const float *bias;
    int sigmoid, n_group, group_size, topk_group, group_top, top_k, renormalise;
    float scale;
    int32_t *ids;
    float *weights;
    int group_lanes, group_magic, smem_words;   // filled in by launch_route
};
cudaError_t launch_route(const RouteParams &p, int sm_count, bool pdl, cudaStream_t s);

// ------------------------------------------------------------------ rounding to 8 bits
cudaError_t launch_quantise_rows(const uint16_t *x, int64_t rows, int64_t K, int64_t ldx, uint8_t *q, int64_t ldq,
                                 float *scales, int sm_count, bool pdl, cudaStream_t s);
cudaError_t launch_quantise_tiles(const uint16_t *x, int64_t rows, int64_t K, int64_t ldx, uint8_t *q, int64_t ldq,
                                  float *scales, bool pdl, cudaStream_t s);

// ------------------------------------------------------------------ dispatch and combine
// A token tile of a grouped product: rows [row0, row0 + rows) of the sorted pairs, one expert.
struct Tile {
    int row0, rows, expert, pad;
};

struct DispatchParams {
    const uint16_t *x;
    int64_t T, H;
    int align;             // of x's rows in bytes, 16 at most
    const int32_t *ids;
    int top_k;
    int64_t first_expert;
    int E;
    int chunk;             // tokens per CTA row (chunk * top_k <= kDispatchPairs)
    int n_chunks, splits;
    int *hist;             // [n_chunks + 1 x E] pairs of each expert before each chunk; null: every CTA counts all ids
    int32_t *pos;          // [T x top_k] row of a pair among the sorted pairs, -1: not of this rank
    Tile *tiles;
    int *n_tiles;
    int tile_rows;
    uint8_t *xq; int64_t ldq;
    float *xs;
};
constexpr int kDispatchThreads = 256;
constexpr int kDispatchPairs = 256;
int align_of(const uint16_t *x, int64_t ld);   // of rows of pitch ld, in bytes, 16 at most
cudaError_t launch_dispatch(const DispatchParams &p, bool pdl, cudaStream_t s);

// y[t] = shared[t] + sum_j w[t, j] o[pos[t, j]]
cudaError_t launch_combine(const float *o, int64_t ldo, const int32_t *pos, const float *weights, int top_k,
                           const uint16_t *shared, uint16_t *y, int64_t T, int64_t H, int sm_count, bool pdl,
                           cudaStream_t s);

// ------------------------------------------------------------------ block-scaled products
constexpr int kRoundRows = 8;

enum BlockEpi : int {
    BLOCK_BF16 = 0,      // out bf16
    BLOCK_F32 = 1,       // out fp32
    BLOCK_SWIGLU = 2,    // silu(g) u: rounded to 8 bits with scales (tensor-core kernels), fp32 (generic)
};

struct BlockGemm {
    // token rows: rows [0, T) of one group (tiles null), or the tiles of a dispatch (T: their rows at most)
    int64_t T;
    const Tile *tiles;
    const int *n_tiles;
    const int32_t *ids;            // at most 32 pairs: the tile of a slot is found from the ids, not the table
    int pairs;
    int64_t first_expert;
    int max_tiles;
    int expected_tiles;            // as the host expects it (chooses grids, not results)
    int tile_rows;
    const uint8_t *xq; int64_t ldx;
    const float *xs;               // [rows x kb]
    const uint16_t *x; int64_t ldxb;   // up to kRoundRows rows of a plain product in bf16, rounded by the product's kernel; or null
    int x_wide;                    // x in 16-byte words
    const uint8_t *wq; int64_t ldw;
    const float *ws;               // [.. x kb] blocks
    int64_t N, K;                  // weight rows of one product (I for SWIGLU), inner size
    int kb;                        // k-blocks
    int groups;                    // experts (1 for a plain product)
    int64_t w_group_rows;          // weight rows of one expert in wq
    int64_t ws_group;              // scales of one expert
    int64_t up_rows, up_scales;    // SWIGLU: from a gate row / scale to its up row / scale
    int epi;
    void *out; int64_t ldo;        // BF16 / F32 (and the generic kernels' SWIGLU, fp32)
    uint8_t *hq; int64_t ldh;      // SWIGLU: rounded h and its scales [rows x hb]
    float *hs; int hb;
    int weights_early;             // the weights are complete before this launch can start (swap-AB kernel)
    uint64_t wait_limit_ns;
    uint32_t *err;
};

// How a product's grid is split: CTAs, and the CTAs (CTA pairs) that share a tile's k-blocks.
struct Split {
    int64_t ctas;
    int parts;
};

// Tensor-core kernel for token tiles of 16, 32 or (not SWIGLU) 64 rows (weights on the 128-row side).
mse_status launch_block_cols(const BlockGemm &g, int sm_count, bool pdl, cudaStream_t s);
int cols_parts(int64_t tiles, int kb, int tile_rows, int epi, int sm_count);
Split cols_split(const BlockGemm &g, int sm_count);
// Tensor-core kernel for token tiles of 256 rows (a CTA pair per 256 x 256 tile).
mse_status launch_block_pair(const BlockGemm &g, int sm_count, bool pdl, cudaStream_t s);
int pair_parts(int64_t tiles, int kb);
Split pair_split(const BlockGemm &g, int sm_count);

constexpr int kSimtTileRows = 16;
cudaError_t launch_block_simt(const BlockGemm &g, bool pdl, cudaStream_t s);
// fp32 rows to 8 bits, as the tensor-core kernels' epilogue does it
cudaError_t launch_quantise_f32(const float *h, const int *n_tiles, const Tile *tiles, int64_t max_tiles, int64_t K,
                                uint8_t *q, int64_t ldq, float *scales, bool pdl, cudaStream_t s);

}  // namespace routed
}  // namespace mse
