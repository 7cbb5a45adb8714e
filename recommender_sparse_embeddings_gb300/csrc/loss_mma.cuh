// The softmax loss's products on the tensor cores (tcgen05): what its kernels
// share, host and device.
//
// All of the loss's work is three kinds of products:
//   scores   S = X W^T            (rows x items, over the D columns)
//   gx       dX += d W            (rows x columns, over the items)
//   gw       dW = d^T X           (items x columns, over the rows)
// The forward pass takes the scores alone; the backward pass all three, up to 256
// columns (fp32: 128) in the fused kernel and above in the step kernel, with d in
// memory.  The forward and the step kernel: a persistent CTA per SM takes work items
// in turn; one warp fetches operand tiles by TMA, one issues the products (128 x up
// to 256, fp32 in tensor memory, two accumulators of 256 columns), and the first 16
// (step kernel: 8) read the accumulators: one item's arithmetic runs under the next
// item's products.  X, W and d lie row by row in memory; the products read them
// K-major or MN-major by the descriptor alone, so nothing is transposed.
//
// fp32.  An fp32 number is the sum of three bf16 numbers exactly (8 bits each,
// rounded to nearest, the rest carried on).  fp32 operands are kept as three
// such planes, and a product is the sum of the six plane products of at least
// 2^-18 of the whole, the small ones first; the three left out are below 2^-26,
// less than an fp32 rounding.
//
// Long sums.  The tensor units cut an fp32 sum at every addition instead of
// rounding it, so long sums drift towards 0: 20,011 items in one accumulator made
// fp32's grad_x 2.2e-5 off, 1,000,000 made fp16's 1.2e-3 off, where its rounding is
// 2.1e-4.  An accumulator is therefore added, rounded, to a sum in memory and begun
// anew every kFlush (fused: kFusedFlush) blocks of 64 along the sum with fp32, whose
// large products (of the first planes) come last or have an accumulator of their
// own, and every kLongSum rows or items with 16-bit types.  A score is such a sum
// too: above 512 columns it is taken in parts of up to kScorePart blocks of 64, which
// are added up in registers (but for the d of 16-bit types, which is rounded to 8 or
// 11 bits: its parts changed no error and took 8 to 12 % of the backward pass).
#pragma once

#include <cuda.h>

#include "attention_mma.cuh"

namespace tbe {

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap& map, int col, int64_t row, int plane,
                                         uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(&map), "r"(col), "r"((int)row), "r"(plane), "r"(smem_u32(bar))
        : "memory");
}

// Eight consecutive elements on a 16-byte boundary.
template <int OUT>
__device__ __forceinline__ void store8(void* out, int64_t at, const float* x) {
    if constexpr (OUT == DT_F32) {
        float4* to = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
        to[0] = make_float4(x[0], x[1], x[2], x[3]);
        to[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
            make_uint4(pack2<OUT>(x[0], x[1]), pack2<OUT>(x[2], x[3]), pack2<OUT>(x[4], x[5]), pack2<OUT>(x[6], x[7]));
    }
}

// The accumulator's chunks of W columns of this warpgroup (one of GROUPS) into
// a slab of partial sums: [columns / 4][128 rows] of float4, so that a warp's
// 32 rows are 512 consecutive bytes.
template <int GROUPS, int W = 32>
__device__ __forceinline__ void add_slab(float4* to, uint32_t acc, int wide, int group, bool first) {
    for (int c = group * W; c < wide; c += W * GROUPS) {
        float x[W];
        if constexpr (W == 32)
            tmem_ld32_issue(acc + c, x);
        else
            tmem_ld16(acc + c, x);
        float4 old[W / 4];
        if (!first) {
#pragma unroll
            for (int q = 0; q < W / 4; ++q) old[q] = to[(c / 4 + q) * 128];
        }
        if (W == 32) tmem_wait_ld(x, W);
#pragma unroll
        for (int q = 0; q < W / 4; ++q) {
            float4 v = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
            if (!first) v.x += old[q].x, v.y += old[q].y, v.z += old[q].z, v.w += old[q].w;
            to[(c / 4 + q) * 128] = v;
        }
    }
}

// The same chunks, times `times`, as columns of the thread's row of a result
// that starts at element `at` and has `left` columns; added to an fp32 result
// where `add` says so.
template <int OUT, int GROUPS>
__device__ __forceinline__ void store_rows(void* out, int64_t at, uint32_t acc, int wide, int group, bool valid,
                                           int left, bool vec, float times, bool add = false) {
    vec = vec && (uintptr_t)out % 16 == 0;
    for (int c = group * 32; c < wide; c += 32 * GROUPS) {
        float x[32];
        tmem_ld32_issue(acc + c, x);
        tmem_wait_ld(x, 32);
        if (!valid) continue;
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] *= times;
        if (OUT == DT_F32 && add) {
            const float* old = static_cast<const float*>(out) + at + c;
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (c + e < left) x[e] += old[e];
        }
        if (vec) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
                if (c + e >= left) break;
                store8<OUT>(out, at + c + e, x + e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (c + e < left) store_elem<OUT>(out, at + c + e, x[e]);
        }
    }
}

// 128 rows x 32 columns of a result: the slabs' sum in order, times `times`,
// rounded; 256 threads.
template <int OUT>
__device__ __forceinline__ void finish(const float4* part, int64_t slab_stride, int slabs, void* out, int64_t row0,
                                       int rows, int D, int col0, float times, int thread) {
    const int r = thread % 128;
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4* from = part + (col0 / 4 + thread / 128 * 4) * 128 + r;
#pragma unroll 4
    for (int s = 0; s < slabs; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 y = from[s * slab_stride + i * 128];
            v[i].x += y.x, v[i].y += y.y, v[i].z += y.z, v[i].w += y.w;
        }
    if (r >= rows) return;
    const int col = col0 + thread / 128 * 16;
    const int64_t at = (row0 + r) * D + col;
    const bool vec = D % 8 == 0 && (uintptr_t)out % 16 == 0;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        float x[8] = {v[i].x,     v[i].y,     v[i].z,     v[i].w,
                      v[i + 1].x, v[i + 1].y, v[i + 1].z, v[i + 1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= times;
        if (vec) {
            if (col + i * 4 >= D) break;
            store8<OUT>(out, at + i * 4, x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col + i * 4 + e < D) store_elem<OUT>(out, at + i * 4 + e, x[e]);
        }
    }
}

constexpr int kLossThreads = 320;
constexpr int kLossStages = 4;
// Blocks between two such additions: the drift grows with them and so does the
// time without (2050 x 20011 x 96 fp32, plain fp32 torch 7.2e-7 off; fused: 4 235 us
// and 4.8e-7, 6 211 us and 6.7e-7, 8 203 us and 8.8e-7, 16 189 us and 1.7e-6).
constexpr int kFlush = 8, kFusedFlush = 6;
// 16-bit types: rows or items, 16 of them a product; a cut loses 2^-25 of the final
// sum on average, so 32,768 drift by 6e-5, a third of fp16's rounding.
// (10,000 x 1,000,000 x 128 f16: 1.18e-3 off without, 2.1e-4 with, 5.39 and 5.34 ms;
// 131,072 x 40,000 x 64 f16: 2.81 and 2.89 ms.)
constexpr int kLongSum = 32768;
// Blocks of 64 columns that a part of the scores has at most (an accumulator's error
// of lse at 4096 columns: in one 8e-7, in parts of 8 1e-7), and has: equal parts.
// Below, the kernels are built without parts (with them they lost 5 % at 512 columns).
constexpr int kScorePart = 8;
__host__ __device__ constexpr int score_part_blocks(int D) {
    const int blocks = (D + 63) / 64, parts = (blocks + kScorePart - 1) / kScorePart;
    return (blocks + parts - 1) / parts;
}
constexpr int kBox = 64 * 64 * 2;  // bytes of a TMA box: 64 columns x 64 rows
constexpr int kStageBytes = 6 * kBox;  // A: 2 boxes, B: 4
constexpr int kStagingBytes = 4096;    // of a warp: 32 rows x 64 columns of d
constexpr int kLossSmem = kLossStages * kStageBytes + 8 * kStagingBytes + 1024;

enum : int32_t { ITEM_GW = 0, ITEM_GX = 1, ITEM_D = 2, ITEM_FIN_W = 3, ITEM_FIN_X = 4 };

// The softmax's arguments.  16-bit types work in base 2 (one multiply-add before
// ex2).  fp32 takes the difference to lse (or to the maximum) in natural units and
// multiplies then: rounding lse log2(e) would move a whole row by 2^-24 of it,
// 1e-6 at a lse of 14, which is more than the rest of fp32's errors.
template <int P>
__device__ __forceinline__ void powers(float& a, float& b, float scale, float less_a, float less_b) {
    fma2(a, b, scale, less_a, less_b);
    if (P == 3) mul2(a, b, kLog2e, kLog2e);
    a = ex2(a);
    b = ex2(b);
}

// What the rows bring into the backward pass: per tile of 128 rows 128 values
// each of -lse (times log2(e) but for fp32; fp16: + 14), of g over the largest |g|,
// of the target as an int32, and of what a row's own sum is multiplied by (g scale;
// fp16: 2^-14 of it); -inf, 1, -1 and 0 in rows that are left out or behind the last.
constexpr int kRowValues = 4 * 128;

// What d has of the target: 1, or with fp16 2^14.
template <int DT>
__host__ __device__ constexpr float target_unit() {
    return DT == DT_F16 ? 16384.f : 1.f;
}

struct LossForward {
    int64_t N, v0, v1;  // rows; the items of this launch
    int64_t w0;         // the item at the table map's first row
    int32_t D, row_tiles, item_tiles, slices;
    int32_t first;  // else the sums go on from `part`
    float c2;       // scale, times log2(e) but for fp32
    const void* targets;
    int32_t index64;
    int64_t V;
    float2* part;   // [N][slices][4]: maximum and sum of a quarter of a slice's columns
    float* picked;  // [N]: the target's logit
    uint32_t* error;
};

// CTAs of a backward launch at most.
constexpr int kMaxStepCtas = 256;

// One launch of the backward pass: d of a piece of the table, the products of
// the piece before it, the results of the piece before that.
struct LossStep {
    int64_t N, V;
    int32_t D, row_tiles, col_tiles;  // col_tiles: of 256 columns
    float c2;
    const float* rows;   // [row_tiles][kRowValues]
    const float* unit;   // what the products of d are multiplied by
    // d of the items from d0 on, its work items d_from[c] .. d_from[c + 1] by CTA c
    int32_t n_d;
    int32_t d_from[kMaxStepCtas + 1];
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

// The work of one gradient in a fused launch: a CTA for each of `tiles` tiles
// of 128 lines and each slice of the `others` tiles along the sum.
struct LossSide {
    int32_t tiles, others, slices;
    int32_t first, last;  // over spans of the table: the sums begin, end here
    int32_t direct;       // a CTA's sums are the result's (fp32: are added there)
    float4* part;         // [slices][tiles][cols4][128] else
    void* out;
};

// Both gradients of operands of up to 256 columns (fp32: 128), d never leaving
// the SM: grad_x's CTAs come first, then grad_table's.
struct LossFused {
    int64_t N, V, v0, v1;  // the call's items and this launch's
    int64_t w0;            // the item at the table map's first row
    int32_t D, cols4;
    float c2;
    const float *rows, *unit;
    LossSide x, w;
    uint32_t* error;
};

struct LossFusedMaps {
    CUtensorMap x, w;
};

// The results whose sums lie in several slabs.
struct LossFinish {
    LossSide x, w;  // tiles 0: nothing to do
    int64_t x_rows, w_rows;
    const float *rows, *unit;
    int32_t D, cols4;
};

cudaError_t loss_mma_configure();
cudaError_t loss_fused_configure();
// Lines of the tiles that the fused kernel walks.
constexpr int loss_fused_walk(int D, int planes) { return D <= 128 && planes == 1 ? 128 : 64; }
// Such tiles that one of its accumulators takes.
constexpr int loss_fused_flush(int D, int planes) {
    return planes == 3 ? kFusedFlush : kLongSum / loss_fused_walk(D, planes);
}
cudaError_t launch_loss_fused(const LossFused& p, const LossFusedMaps& maps, int dtype, cudaStream_t s);
cudaError_t launch_loss_finish(const LossFinish& p, int dtype, cudaStream_t s);
cudaError_t launch_loss_forward(const LossForward& p, const LossMaps& maps, int dtype, int grid, cudaStream_t s);
cudaError_t launch_loss_step(const LossStep& p, const LossMaps& maps, int dtype, int grid, cudaStream_t s);

}  // namespace tbe
