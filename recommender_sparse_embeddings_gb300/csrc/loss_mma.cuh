// The softmax loss's products on the tensor cores (tcgen05): what its kernels
// share, host and device.
//
// All of the loss's work is three kinds of products:
//   scores   S = X W^T            (rows x items, over the D columns)
//   gx       dX += d W            (rows x columns, over the items)
//   gw       dW = d^T X           (items x columns, over the rows)
// and one kernel runs them all.  A persistent CTA per SM takes work items in
// turn; warp 8 fetches operand tiles by TMA, warp 9 issues the products (128 x
// up to 256, fp32 in tensor memory, two accumulators of 256 columns), warps 0
// to 7 read the accumulators: one item's arithmetic runs under the next item's
// products.  X, W and d lie row by row in memory; the products read them
// K-major or MN-major by the descriptor alone, so nothing is transposed.
//
// fp32.  An fp32 number is the sum of three bf16 numbers exactly (8 bits each,
// rounded to nearest, the rest carried on).  fp32 operands are kept as three
// such planes, and a product is the sum of the six plane products of at least
// 2^-18 of the whole, added small ones first; the three left out are below
// 2^-26, less than an fp32 rounding.
#pragma once

#include <cuda.h>

#include "attention_mma.cuh"

namespace tbe {

constexpr int kLossThreads = 320;
constexpr int kLossStages = 4;
constexpr int kBox = 64 * 64 * 2;  // bytes of a TMA box: 64 columns x 64 rows
constexpr int kStageBytes = 6 * kBox;  // A: 2 boxes, B: 4
constexpr int kStagingBytes = 4096;    // of a warp: 32 rows x 64 columns of d
constexpr int kLossSmem = kLossStages * kStageBytes + 8 * kStagingBytes + 1024;

enum : int32_t { ITEM_GW = 0, ITEM_GX = 1, ITEM_D = 2, ITEM_FIN_W = 3, ITEM_FIN_X = 4 };

// What a row brings into the backward pass.
struct RowStat {
    float minus_lse2;  // -lse log2(e); 0 in rows left out
    float coef;        // g * scale; 0 in rows left out
    int32_t target;    // -1 in rows left out
    int32_t pad;
};

struct LossForward {
    int64_t N, v0, v1;  // rows; the items of this launch
    int64_t w0;         // the item at the table map's first row
    int32_t D, row_tiles, item_tiles, slices;
    int32_t first;  // else the sums go on from `part`
    float c2;       // scale * log2(e)
    const void* targets;
    int32_t index64;
    int64_t V;
    float2* part;   // [N][2 slices]: maximum and sum (base 2) of a half of a slice's columns
    float* picked;  // [N]: the target's logit (base 2)
    uint32_t* error;
};

// One launch of the backward pass: d of a piece of the table, the products of
// the piece before it, the results of the piece before that.
struct LossStep {
    int64_t N, V;
    int32_t D, row_tiles, col_tiles;  // col_tiles: of 256 columns
    float c2;
    const RowStat* rows;
    const float* gmax;  // fp16: partial maxima of |coef|
    int32_t n_gmax;
    // d of the items from d0 on
    int32_t n_d;
    int64_t d0, dw0;  // dw0, pw0: the items at the first row of the maps w and pw
    // products of the piece [p0, p0 + p_items)
    int32_t n_gx, n_gw;
    int64_t p0, pw0;
    int32_t p_items, first;    // first: gx's sums begin here
    int32_t x_slabs, w_slabs;  // parts of the sums over the items and over the rows
    float4* x_part;            // [x_slabs][row_tiles][cols4][128]
    float4* w_part;            // [w_slabs][tiles of 128 items][cols4][128]; one slab goes to gw at once
    // results
    int32_t n_fin_w, n_fin_x;
    int64_t f0;
    int32_t f_items;
    const float4* f_part;
    void *gx, *gw;
    int32_t cols4;
    uint32_t* error;
};

// The table has two maps: of the piece whose d is computed and of the one
// whose products are (the same unless the table is copied in spans).
struct LossMaps {
    CUtensorMap x, w, pw, d_in, d_out;
};

cudaError_t loss_mma_configure();
cudaError_t launch_loss_forward(const LossForward& p, const LossMaps& maps, int dtype, int grid, cudaStream_t s);
cudaError_t launch_loss_step(const LossStep& p, const LossMaps& maps, int dtype, int grid, cudaStream_t s);

}  // namespace tbe
