// Attention over ragged user histories: what its kernels share.
//
// A history is a run of L tokens; query i and key j of one history, with
// distance d = i - j, see each other when
//     0 <= d  and  (d < window  or  j < sinks)
// and their logit is scale * q_i . k_j + bias[bucket(d)].  All kernels work
// in base 2: logits are multiplied by log2(e) so that the softmax's
// exponential is one ex2, and the saved statistic is
//     lse_i = log2 sum_j 2^(logit_ij * log2 e).
//
// Biases of large magnitude.  A bias of -1e9 on all keys that a row sees must
// not change its weights, but fp32 holds no logit beside it (steps of 128 in
// base 2), nor log2 of the sum in lse.  So the forward takes the largest bias
// that the row sees off each one first (attn_bias_top; only for heads with an
// entry from kCoarse on), and the backward adds up a row's recomputed weights
// 2^(logit - lse) where |lse| is kCoarse or more and divides by their sum
// (its log2 is the row's `excess`).
#pragma once

#include <float.h>
#include <limits.h>

#include "tbe_internal.cuh"

namespace tbe {

constexpr float kLog2e = 1.4426950408889634f;
// Limits of a handle (decode keeps the buckets of eight heads in shared memory).
constexpr int kMaxBuckets = 256;
constexpr int kMaxDistance = 65535;
constexpr int kMaxSinks = 128;
constexpr int kMaxHeadDim = 256;

// Rows of one tensor operand: row (token, head) starts at
// data + token * token_stride + head * head_stride (elements).
struct Rows {
    const void* data;
    int64_t token_stride;
    int64_t head_stride;
};

// One tile of one history (a work item of the forward and backward kernels).
struct AttnItem {
    int32_t start;  // the history's first token in the batch
    int32_t len;    // its tokens
    int32_t tile;   // the tile's number, counted from the history's start
    int32_t tiles;  // tiles of the history
};

// The first key tile of a long history with sinks is seen by every query
// behind the window: its far queries, in chunks of blocks, are work items of
// their own (FarItem), which leave fp32 sums of the sinks' rows to a join.
struct FarItem {
    int32_t start, len;
    int32_t chunk, chunks;  // this chunk of the history's far query blocks
    int32_t slot;           // of the history's first partial sums: the tile's own; chunk c has slot + 1 + c
    int32_t pad[3];
};

struct FarWork {
    FarItem* items;
    int32_t* n_items;
    int32_t* slot_of;  // per tile item: its history's first slot, -1 for none
    float* part;       // [slots, Hk, 2, sinks, DP]: dk (unscaled) and dv of the sinks' rows
    int32_t most;      // items at most (0: no history is split)
    int32_t blocks;    // query blocks of 64 a chunk
    int32_t near;      // query blocks of the tile's own item
};

// First words of the handle's device block; the bucket map follows.
struct AttnBlock {
    uint32_t error;  // sticky ERR_* bits
    uint32_t pad[3];
    // uint16_t bucket_of[far + 1]
};

struct AttnShape {
    int32_t dtype;
    int32_t H, Hk, G;  // query heads, key-value heads, query heads per key-value head
    int32_t D;
    int32_t window;  // INT_MAX / 2 where every earlier token is visible
    int32_t sinks;
    int32_t buckets;  // 0: no bias
    int32_t far;      // first distance of the last bucket
    float scale;
    const uint16_t* bucket_of;  // device [far + 1]
    const int32_t* starts;      // device [buckets + 1], ending with INT_MAX
    uint32_t* error;            // device
};

// Where a kernel finds its work items: in the list that the items kernel left,
// or, for a batch of few histories, in the offsets themselves (each warp adds
// up the histories' tiles; a launch of its own costs more than that).
constexpr int kScanHistories = 128;

struct ItemSource {
    const AttnItem* items;
    const int32_t* n_items;
    const void* offsets;  // null: the list
    int64_t N;
    int32_t index64, B, tile;
    uint32_t* error;
};

// Item w of the batch; false if there is none.  All lanes of a warp call it
// together.
__device__ __forceinline__ bool find_item(const ItemSource& s, int64_t w, AttnItem& it) {
    if (!s.offsets) {
        if (w >= *s.n_items) return false;
        it = s.items[w];
        return true;
    }
    const int lane = threadIdx.x % 32;
    int64_t base = 0;
    for (int b0 = 0; b0 < s.B; b0 += 32) {
        const int b = b0 + lane;
        int64_t lo = 0, hi = 0;
        if (b < s.B) {
            lo = s.index64 ? static_cast<const int64_t*>(s.offsets)[b] : static_cast<const int32_t*>(s.offsets)[b];
            hi = s.index64 ? static_cast<const int64_t*>(s.offsets)[b + 1]
                           : static_cast<const int32_t*>(s.offsets)[b + 1];
            const bool bad = lo < 0 || hi < lo || hi > s.N;
            if (bad || (b == 0 && lo != 0) || (b == s.B - 1 && hi != s.N)) atomicOr(s.error, ERR_OFFSETS);
            if (bad) hi = lo = 0;
        }
        const int n = (int)((hi - lo + s.tile - 1) / s.tile);
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, w < base + incl);
        if (hit) {
            const int k = __ffs(hit) - 1;
            const int nk = __shfl_sync(0xffffffffu, n, k), ik = __shfl_sync(0xffffffffu, incl, k);
            const int lk = (int)__shfl_sync(0xffffffffu, lo, k), hk = (int)__shfl_sync(0xffffffffu, hi, k);
            it = AttnItem{lk, hk - lk, (int)(base + ik - 1 - w), nk};  // the history's last tile first
            return true;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
}

// Items of the batch, by the same rules.
__device__ __forceinline__ int64_t count_items(const ItemSource& s) {
    if (!s.offsets) return *s.n_items;
    const int lane = threadIdx.x % 32;
    int64_t n = 0;  // (overlapping offsets: up to half the histories of N tokens each)
    for (int b = lane; b < s.B; b += 32) {
        const int64_t lo = s.index64 ? static_cast<const int64_t*>(s.offsets)[b] : static_cast<const int32_t*>(s.offsets)[b];
        const int64_t hi = s.index64 ? static_cast<const int64_t*>(s.offsets)[b + 1]
                                     : static_cast<const int32_t*>(s.offsets)[b + 1];
        if (lo >= 0 && hi >= lo && hi <= s.N) n += (hi - lo + s.tile - 1) / s.tile;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n;
}

struct AttnForward {
    AttnShape s;
    Rows q, k, v;
    const void* bias;  // [buckets, H] of dtype, or null
    void* out;         // [N, H, D]
    float* lse;        // [H, N]
    int64_t N;
    ItemSource src;
    int64_t max_items;  // room of the list
    int32_t ctas;  // > 0: so many CTAs take the items in turn; 0: a CTA per item
    int32_t vec;  // rows are 16-byte aligned and D * element size is a multiple of 16
};

struct AttnBackward {
    AttnShape s;
    Rows q, k, v, g;
    const void* bias;
    const void* out;   // [N, H, D]
    const float* lse;  // [H, N]
    void* gq;          // [N, H, D]
    void* gk;          // [N, Hk, D]
    void* gv;          // [N, Hk, D]
    float* delta;      // workspace [H, N]: g_i . out_i
    float* size;       // workspace [H, N], fp16 on the tensor cores: the largest |element| of g_i
    float* excess;     // workspace [H, N], where |lse| >= kCoarse: log2 of the sum of 2^(logit - lse)
    float* bias_part;  // workspace [items, then far items, H, buckets]
    int64_t max_items;
    FarWork far;
    int64_t N;
    ItemSource src;
    int32_t vec;
};

// Division by a number fixed per launch, for x < 2^31: with c = ceil(log2 n)
// and m = ceil(2^(31 + c) / n) < 2^32, the error x * (m - 2^(31+c)/n) / 2^(31+c)
// is below x / 2^(31+c) <= 1 / n, so x * m >> (31 + c) is the floor.
struct FastDiv {
    uint32_t n, m, s;
};

inline FastDiv make_fast_div(uint32_t n) {
    uint32_t c = 0;
    while ((uint64_t(1) << c) < n) ++c;
    const uint64_t p = uint64_t(1) << (31 + c);
    return FastDiv{n, (uint32_t)((p + n - 1) / n), 31 + c};
}

__host__ __device__ __forceinline__ uint32_t fast_div(uint32_t x, FastDiv d) {
    return (uint32_t)(((uint64_t)x * d.m) >> d.s);
}

struct AttnDecode {
    AttnShape s;
    Rows q;            // token = history of the batch
    const void* kp;    // pages: row (page, token, head)
    const void* vp;
    int64_t k_page, k_token, k_head, v_page, v_token, v_head;  // strides (elements)
    const int32_t* table;  // [B, width]
    const int32_t* lengths;
    const void* bias;
    void* out;  // [B, H, D]
    float* part;  // workspace [B, H, splits, D + 2] (D sums, max, sum of weights)
    int32_t width, num_pages, B, chunk, splits;
    int64_t max_length;
    FastDiv page;
    int32_t vec;
};

struct AttnAppend {
    int32_t Hk, D, e;  // e: element bytes
    Rows k, v;
    const void* offsets;
    int32_t index64;
    const int32_t* before;
    void* kp;
    void* vp;
    int64_t k_page, k_token, k_head, v_page, v_token, v_head;
    const int32_t* table;
    int32_t width, num_pages, B;
    int64_t N;
    FastDiv page;
    uint32_t* error;
    int32_t vec;
};

// 2^x by the special-function unit (relative error about 2^-22; 2^-inf = 0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A bias entry in base 2.  The product of a type's lowest finite value with
// log2(e) leaves fp32's range; it is held at fp32's lowest instead (its
// largest at fp32's largest), so a row whose visible keys all carry it keeps
// equal weights (an entry of -inf stays -inf and hides its keys).
__device__ __forceinline__ float bias_base2(float b) {
    const float x = b * kLog2e;
    return fabsf(b) <= FLT_MAX ? fminf(fmaxf(x, -FLT_MAX), FLT_MAX) : x;
}

__device__ __forceinline__ int attn_bucket(const AttnShape& s, int d) {
    return d >= s.far ? s.buckets - 1 : (int)__ldg(s.bucket_of + d);
}

// From this magnitude on (base 2) a bias or a row's statistic is kept apart
// from the logits: below it the sum with a logit of its size is off by 2^-18 at
// most, 3e-6 of a weight.
constexpr float kCoarse = 64.f;

// Neither an infinity nor a type's lowest value counts: they hide their keys
// exactly.
__device__ __forceinline__ bool attn_coarse(float x) { return fabsf(x) >= kCoarse && fabsf(x) <= FLT_MAX && x > -FLT_MAX; }

// The largest bias (base 2) of the keys that query i sees, over every `step`-th
// bucket from `at` on of those that its distances have: 0 .. min(i, window - 1),
// and behind the window the sinks' i - sinks + 1 .. i.  bias_of(b): bucket b's.
template <typename F>
__device__ __forceinline__ float attn_bias_top(const AttnShape& s, int i, int at, int step, F bias_of) {
    float top = -INFINITY;
    const int near = attn_bucket(s, tmin(i, s.window - 1));
#pragma unroll 1
    for (int b = at; b <= near; b += step) top = fmaxf(top, bias_of(b));
    if (i >= s.window && s.sinks > 0) {
        const int last = attn_bucket(s, i);
#pragma unroll 1
        for (int b = attn_bucket(s, tmax(s.window, i - s.sinks + 1)) + at; b <= last; b += step)
            top = fmaxf(top, bias_of(b));
    }
    return top;
}

// What is taken off the row's biases, given their largest: nothing where the
// row sees no key, or only keys of the lowest value (its logits are then
// swallowed and its weights equal).
__device__ __forceinline__ float attn_bias_off(float top) { return fabsf(top) <= FLT_MAX && top > -FLT_MAX ? top : 0.f; }

__device__ __forceinline__ bool attn_visible(int d, int j, int window, int sinks) {
    return d >= 0 && (d < window || j < sinks);
}

// A saved statistic of a row that has no weights to pass gradients through: it
// sees nothing (-inf), or all it sees carries a bias of its type's lowest
// value, which swallowed the logits.
__device__ __forceinline__ bool attn_no_weights(float lse) { return lse <= -FLT_MAX; }

// The power of two that brings x, the largest |element| of upstream gradients
// in fp16, into [4, 8): at an ordinary scale about 1, so that small logits'
// gradients keep the bits they have there, and 2^13 below fp16's largest, for
// the sum over a value row.  1 for 0, infinities and NaN.
__device__ __forceinline__ float attn_unit(float x) {
    const uint32_t e = __float_as_uint(x) & 0x7f800000u;
    return e < 0x01000000u || e >= 0x7f000000u ? 1.f : __uint_as_float(0x7f000000u + 0x01000000u - e);
}

// Its inverse.
__device__ __forceinline__ float attn_unit_back(float s) { return __uint_as_float(0x7f000000u - __float_as_uint(s)); }

// Whether key j is the only one that query i can see.  Its weight is 1
// whatever the logit, so the logit's gradient is exactly 0, which dp - delta,
// two sums of the same products in different orders, would miss by rounding.
__device__ __forceinline__ bool attn_lone(int i, int j, int window, int sinks) {
    return i == j && (i == 0 || (window == 1 && sinks == 0));
}

template <int DT>
struct Elem;
template <>
struct Elem<DT_F32> {
    using type = float;
};
template <>
struct Elem<DT_F16> {
    using type = __half;
};
template <>
struct Elem<DT_BF16> {
    using type = __nv_bfloat16;
};

struct AttnMaps;

// Launchers (each returns the launch's status).
cudaError_t launch_attn_items(const void* offsets, int index64, int64_t N, int B, int tile, AttnItem* items,
                              int64_t capacity, int32_t* n_items, uint32_t* error, const FarWork& far,
                              cudaStream_t s);
cudaError_t launch_attn_forward_simt(const AttnForward& p, int64_t max_items, cudaStream_t s);
cudaError_t launch_attn_backward_simt(const AttnBackward& p, int64_t max_items, cudaStream_t s);
cudaError_t launch_attn_forward_mma(const AttnForward& p, const AttnMaps& maps, cudaStream_t s);
cudaError_t attn_forward_mma_configure();
cudaError_t launch_attn_backward_mma(const AttnBackward& p, const AttnMaps& maps, int64_t max_items, cudaStream_t s);
cudaError_t attn_backward_mma_configure();
cudaError_t launch_attn_bias_reduce(const AttnBackward& p, void* grad_bias, cudaStream_t s);
cudaError_t launch_attn_append(const AttnAppend& p, cudaStream_t s);
cudaError_t launch_attn_decode(const AttnDecode& p, cudaStream_t s);
cudaError_t attn_simt_configure(int optin_smem);
int attn_simt_tile(int dtype, int D, int H, int64_t N, int64_t B, int num_sms);
// query heads one decode CTA takes at once
int attn_decode_heads(int G);

}  // namespace tbe
