// Internal interfaces of the sorted rows (tokens sorted by expert and back) and of the products in 8-bit integers.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mse.h"

namespace mse {
namespace sorted {

constexpr int64_t kMaxRows = (int64_t)1 << 30;     // rows and columns: indexes of rows stay in 32 bits
constexpr int64_t kMaxInner = (int64_t)1 << 22;
constexpr int64_t kMaxPitch = (int64_t)1 << 32;
constexpr int64_t kMaxInt8Inner = ((int64_t)1 << 17) - 1;   // 2^14 K stays below 2^31

// ------------------------------------------------------------------ tokens sorted by expert
constexpr int kSortThreads = 256;                  // and at most as many pairs to a chunk of tokens

struct SortParams {
    const uint8_t *x; int64_t T, row_bytes, ldx;   // ldx, ldr: bytes
    const int32_t *ids;
    int top_k;
    int64_t first_expert;
    int E;
    const float *scales;                           // [T] or null
    uint8_t *rows; int64_t ldr;
    float *row_scales;
    int32_t *place, *offsets;
    int chunk, n_chunks;                           // tokens of a CTA row (chunk * top_k <= kSortThreads)
    int splits;                                    // CTAs that share a chunk's copies
    int few;                                       // few bytes in all: a warp copies one word a lane at a time
    int *hist;                                     // [n_chunks + 1 x E], or null: every CTA counts all ids
    int unit;                                      // bytes of a copied word: divides every address and row_bytes
};
cudaError_t launch_sort(const SortParams &p, bool pdl, cudaStream_t s);

// ------------------------------------------------------------------ and back
struct UnsortParams {
    const void *rows; int64_t n_rows, ldr;         // pitch in elements
    const int32_t *place;
    const float *weights;                          // [T x top_k] or null: 1
    int top_k;
    const void *base;                              // [T x H] of y's type, or null: 0
    void *y;
    int64_t T, H;
    int rows_f32, y_f32;
};
cudaError_t launch_unsort(const UnsortParams &p, int sm_count, bool pdl, cudaStream_t s);

struct UnsortBackwardParams {
    const void *dy;                                // [T x H]
    const int32_t *place;
    const float *weights;                          // or null: 1, and no dweights
    const void *rows; int64_t ldr;                 // or null
    int top_k;
    void *drows; int64_t ldd, n_rows;
    float *dweights;
    int64_t T, H;
    int dy_f32, rows_f32;
};
cudaError_t launch_unsort_backward(const UnsortBackwardParams &p, int sm_count, bool pdl, cudaStream_t s);

// ------------------------------------------------------------------ 8-bit integers
struct RoundParams {
    const void *x; int64_t rows, K, ldx;           // pitch in elements; swiglu: [rows x 2K], gate before up
    int f32, swiglu;
    const int32_t *last;                           // rows from *last on are left alone; null: none is
    void *q; int64_t ldq;                          // int8, or the same integers in fp16 (pitch in elements)
    int half_out;
    float *scales;
};
cudaError_t launch_int8_round(const RoundParams &p, int sm_count, bool pdl, cudaStream_t s);

struct Int8Gemm {
    int64_t T;                                     // token rows (grouped: at most)
    const int8_t *xq; int64_t ldx;                 // int8 rows (generic kernels)
    const uint16_t *x16; int64_t ldx16;            // the same integers in fp16 (tensor-core kernels)
    const float *xs;
    const int32_t *offsets;                        // grouped: [groups + 1], else null
    int groups;
    const int8_t *wq; int64_t ldw;                 // [groups * N x K]
    const float *ws;                               // [groups * N]
    int64_t N, K;
    void *out;                                     // [T x N]
    int out_f32;
    uint64_t wait_limit_ns;
    uint32_t *err;
};
cudaError_t launch_int8_simt(const Int8Gemm &g, bool pdl, cudaStream_t s);
// int8 rows to the same integers in fp16; rows from *last on are left out
cudaError_t launch_int8_expand(const int8_t *x, int64_t ldx, int64_t rows, int64_t K, const int32_t *last, uint16_t *out,
                               int64_t ldo, int sm_count, bool pdl, cudaStream_t s);
// Kernel for token tiles of 1, 2 or 4 rows, whose tokens fit kInt8FewBytes of shared memory; with x (bf16 or fp32, of a plain
// product of one row) it rounds the token itself.
constexpr int kInt8FewBytes = 100 * 1024;
bool int8_few_serves(int tile_rows, int64_t K);
cudaError_t launch_int8_few(const Int8Gemm &g, int tile_rows, const void *x, int f32, int64_t ldx, bool weights_early, int sm_count,
                            bool pdl, cudaStream_t s);
// Tensor-core kernel for token tiles of 16, 32 or 64 rows (weights on the 128-row side).
mse_status launch_int8_cols(const Int8Gemm &g, int tile_rows, int sm_count, bool pdl, cudaStream_t s);
// Tensor-core kernel for token tiles of 256 rows (a CTA pair per 256 x 256 tile).
mse_status launch_int8_pair(const Int8Gemm &g, int sm_count, bool pdl, cudaStream_t s);
int int8_pair_parts(int64_t tiles, int kb);
int64_t int8_pair_tiles(const Int8Gemm &g);                  // tiles at most
int int8_cols_parts(int64_t tiles, int kb, int sm_count);
int64_t int8_cols_slots(const Int8Gemm &g, int tile_rows);   // token tiles at most

}  // namespace sorted
}  // namespace mse
