// Tensor-core building blocks of the attention kernels: tiles of 16-bit rows
// in shared memory, operands in tensor memory, and bounded waits.
//
// Tiles.  A tile of R rows (tokens) of DP columns is stored as DP / 64 slabs
// of R rows x 128 bytes in the 128-byte swizzle: 16-byte chunk c of row r at
// chunk c ^ (r & 7).  One copy serves as a K-major operand (the product runs
// over the columns: Q K^T) and as an MN-major one (over the rows: P V), by
// its descriptor alone, so nothing is transposed.
#pragma once

#include <cuda.h>

#include "attention.cuh"
#include "tcgen05.cuh"

namespace tbe {

// Bounded wait: a plain test first (a phase that has completed is the usual
// case), then tries that may each suspend the thread up to the hint (about 2
// us), so 2^20 of them end within seconds.
__device__ __forceinline__ bool mbar_wait_tight(uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    if (ok) return true;
    for (int i = 0; i < kSpinLimit; ++i) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(a), "r"(parity), "r"(2000u)
            : "memory");
        if (ok) return true;
    }
    return false;
}

// The bias of every distance in shared memory, in base 2: entry x belongs to
// distance x - 127, for distances up to `far` and a block's width beyond, or
// up to `most` where the CTA sees no larger ones.  Kept where `far` is at most
// kWholeFar (9 KB); filling it once per CTA (and head) is hidden behind the
// first tiles' fetch, where a table per block by one warp held up every block
// that had several buckets (long window f16: 280 us forward, the softmax
// waiting 1500 to 2300 of its 3900 cycles a block).
constexpr int kWholeFar = 2047;
constexpr int kWholeEntries = kWholeFar + 191 + 127 + 3;

// Returns whether the thread saw an entry of large magnitude.
template <int DT>
__device__ __forceinline__ bool fill_bias(float* table, const AttnShape& s, const void* bias, int head, int most,
                                          int thread, int threads) {
    const int n = tmin(s.far + 190, most) + 128;
    float size = 0.f;
#pragma unroll 4
    for (int x = thread; x < n; x += threads) {
        const int d = x - 127;
        const float b = d >= 0 ? bias_base2(load_elem<DT>(bias, (int64_t)attn_bucket(s, d) * s.H + head)) : 0.f;
        table[x] = b;
        size = fmaxf(size, fabsf(b));
    }
    bool large = size >= kCoarse;
    if (large) {  // not if they are infinities and lowest values
        large = false;
        for (int x = thread; x < n; x += threads) large |= attn_coarse(table[x]);
    }
    return large;
}

// Whether the table of all distances is kept: by the handle's buckets alone, so
// that all heads agree. It shares its memory with the tables per block, which
// the helper warp writes two blocks, heads and turns ahead of the arithmetic.
__device__ __forceinline__ bool keep_whole(const AttnShape& s) { return s.far <= kWholeFar; }

// The last bucket's bias of a head, in base 2.
template <int DT>
__device__ __forceinline__ float last_bias_of(const AttnShape& s, const void* bias, int head) {
    return bias ? bias_base2(load_elem<DT>(bias, (int64_t)(s.buckets - 1) * s.H + head)) : 0.f;
}

// Descriptor of an MN-major operand in the tile layout: 8-row groups (along
// K) are 1024 bytes apart, 64-column blocks (along M or N) one slab.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr, uint32_t slab) {
    return smem_desc(addr, slab, 1024u) | ((uint64_t)2u << 61);
}

// True in one lane of a converged warp.  The products are issued under this
// election by a warp whose other lanes run along: the compiler then knows the
// operands to be uniform (under a plain `lane == 0` each issue took about a
// hundred cycles, and the products' issue bounded the kernels).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// D[tmem] = A B^T of K-major tiles, 16 columns a step: A of 128 rows, B of 64.
template <int DP>
__device__ __forceinline__ void issue_scores(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, int ksteps) {
#pragma unroll
    for (int k = 0; k < DP / 16; ++k)
        if (k < ksteps)
            mma_f16(d_tmem, a + (k / 4) * (128 * 128 / 16) + (k % 4) * 2, b + (k / 4) * (64 * 128 / 16) + (k % 4) * 2,
                    idesc, k > 0);
}

// Bit of the instruction descriptor that makes B MN-major.
constexpr uint32_t kMnMajorB = 1u << 16;

// D[tmem] (+)= A[tmem] B[smem]: A's lane is its row, each 32-bit column two
// consecutive 16-bit elements.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// D[tmem] (+)= A B of a 16-bit A in tensor memory (128 x 64, 32 columns, with
// GAP columns left out after the first 16) and a 64-row tile read MN-major.
template <int GAP = 0>
__device__ __forceinline__ void issue_product(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                              bool accumulate) {
#pragma unroll
    for (int k = 0; k < 4; ++k) mma_f16_ts(d_tmem, a_tmem + k * 8 + (k / 2) * GAP, b + k * (2048 / 16), idesc, accumulate || k > 0);
}

// 32 consecutive columns of the thread's lane (no wait).
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
        : "memory");
}

// A later read of a tcgen05.ld's registers stays behind this wait: the
// registers pass through it.
__device__ __forceinline__ void tmem_wait_ld(float* v, int n) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < n; ++i) asm volatile("" : "+f"(v[i]));
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 columns at each of two places of the thread's lane.
__device__ __forceinline__ void tmem_ld16_pair(uint32_t a, uint32_t b, float (&x)[16], float (&y)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]),
          "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
        : "r"(a)
        : "memory");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(y[0]), "=f"(y[1]), "=f"(y[2]), "=f"(y[3]), "=f"(y[4]), "=f"(y[5]), "=f"(y[6]), "=f"(y[7]), "=f"(y[8]),
          "=f"(y[9]), "=f"(y[10]), "=f"(y[11]), "=f"(y[12]), "=f"(y[13]), "=f"(y[14]), "=f"(y[15])
        : "r"(b)
        : "memory");
    tmem_wait_ld(x, 16);
    tmem_wait_ld(y, 16);
}

// Two floats rounded to the 16-bit type, the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if constexpr (DT == DT_BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
    asm("{\n\t.reg .b64 p, q;\n\t"
        "mov.b64 p, {%0, %1};\n\t"
        "mov.b64 q, {%2, %3};\n\t"
        "add.rn.f32x2 p, p, q;\n\t"
        "mov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}

__device__ __forceinline__ void mul2(float& a0, float& a1, float b0, float b1) {
    asm("{\n\t.reg .b64 p, q;\n\t"
        "mov.b64 p, {%0, %1};\n\t"
        "mov.b64 q, {%2, %3};\n\t"
        "mul.rn.f32x2 p, p, q;\n\t"
        "mov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}

// (a0, a1) = (a0, a1) * m + (b0, b1)
__device__ __forceinline__ void fma2(float& a0, float& a1, float m, float b0, float b1) {
    asm("{\n\t.reg .b64 p, q, r;\n\t"
        "mov.b64 p, {%0, %1};\n\t"
        "mov.b64 q, {%2, %2};\n\t"
        "mov.b64 r, {%3, %4};\n\t"
        "fma.rn.f32x2 p, p, q, r;\n\t"
        "mov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(m), "f"(b0), "f"(b1));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A tensor's TMA map: dimensions (column, head, token), or (column, token,
// head) where the heads are the outer ones; boxes of 64 columns x 64 tokens of
// one head in the 128-byte swizzle.  Columns from D on and tokens from N on
// read as zeros.
struct TileMap {
    CUtensorMap map;
    int32_t heads_outer;
};

struct AttnMaps {
    TileMap q, k, v, g;
};

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void tma_load(uint32_t dst, const TileMap& map, int col, int head, int token,
                                         uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(&map.map), "r"(col), "r"(map.heads_outer ? token : head), "r"(map.heads_outer ? head : token),
        "r"(smem_u32(bar))
        : "memory");
}

// A tile of ROWS rows from row `row0` of a history, by one warp; `full`
// completes when it has landed.  Where it reaches past the history's end (its
// last tile only) the rows there belong to the next history: the tile lands
// on `fix`, the warp clears them, and then arrives on `full` itself, so what
// another history holds (a NaN too) never meets a product.
template <int ROWS, int DP>
__device__ __forceinline__ bool load_tile(unsigned char* dst, const TileMap& map, const AttnItem& it, int head,
                                          int row0, uint64_t* full, uint64_t* fix, uint32_t& fix_phase, int lane) {
    const bool part = it.len - row0 < ROWS;
    if (elect_one()) {
        uint64_t* bar = part ? fix : full;
        mbar_expect_tx(bar, ROWS * DP * 2);
        const uint32_t to = smem_u32(dst);
#pragma unroll
        for (int slab = 0; slab < DP / 64; ++slab)
#pragma unroll
            for (int r = 0; r < ROWS; r += 64)
                tma_load(to + slab * (ROWS * 128) + r * 128, map, slab * 64, head, it.start + row0 + r, bar);
    }
    if (!part) return true;
    const bool ok = mbar_wait_tight(fix, fix_phase);
    fix_phase ^= 1u;
    if (!__all_sync(0xffffffffu, ok)) return false;
    for (int slab = 0; slab < DP / 64; ++slab)
        for (int c = (it.len - row0) * 8 + lane; c < ROWS * 8; c += 32)
            *reinterpret_cast<uint4*>(dst + slab * (ROWS * 128) + c * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(full);
    return true;
}

// A loader warp's ring: `steps` tiles of 64 rows through STAGES stages, the
// ring's tiles `base` on; place(n) gives tile n's first row and head.
template <int DP, int STAGES, typename F>
__device__ __forceinline__ bool load_ring(unsigned char* ring, const TileMap& map, const AttnItem& it,
                                          uint64_t* full, uint64_t* empty, uint64_t* fix, uint32_t& fix_phase,
                                          int steps, int lane, F place, int base = 0) {
    for (int n = 0; n < steps; ++n) {
        const int st = (base + n) % STAGES;
        bool ok = base + n < STAGES || mbar_wait_tight(&empty[st], (((base + n) / STAGES) - 1) & 1);
        const int2 at = place(n);
        ok = __all_sync(0xffffffffu, ok) &&
             load_tile<64, DP>(ring + st * (64 * DP * 2), map, it, at.y, at.x, &full[st], fix, fix_phase, lane);
        if (!ok) return false;
    }
    return true;
}

// The warp's 32 rows (row0 ..) of a 128-row tile in shared memory to rows of
// a contiguous [N, heads, D] tensor; rows from `len` on are left out.
template <int DP>
__device__ __forceinline__ void store_tile_rows(void* out, const unsigned char* tile, int row0, int64_t token0,
                                                int first, int len, int heads, int head, int D, int lane) {
    const int chunks = D / 8;
    for (int x = lane; x < 32 * chunks; x += 32) {
        const int r = row0 + x / chunks, ch = x % chunks;
        if (first + r >= len) continue;
        const uint4 u =
            *reinterpret_cast<const uint4*>(tile + (ch / 8) * (128 * 128) + r * 128 + (((ch % 8) ^ (r & 7)) << 4));
        uint16_t* to = static_cast<uint16_t*>(out) + ((token0 + first + r) * heads + head) * D + ch * 8;
        *reinterpret_cast<uint4*>(to) = u;
    }
}

// 32 columns (from c) of the thread's accumulator row, times `mul`, rounded
// into row `row` of a 128-row tile in shared memory.  A second accumulator,
// if there is one, is added first, times `times`.
template <int DT>
__device__ __forceinline__ void tmem_to_tile(unsigned char* tile, uint32_t taddr, int c, int row, float mul,
                                             uint32_t second = 0xffffffffu, float times = 0.f) {
    float o[32];
    tmem_ld32_issue(taddr + c, o);
    tmem_wait_ld(o, 32);
    if (second != 0xffffffffu) {
        float r[32];
        tmem_ld32_issue(second + c, r);
        tmem_wait_ld(r, 32);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = fmaf(times, r[e], o[e]);
    }
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
        uint4 u;
        u.x = pack2<DT>(o[e] * mul, o[e + 1] * mul);
        u.y = pack2<DT>(o[e + 2] * mul, o[e + 3] * mul);
        u.z = pack2<DT>(o[e + 4] * mul, o[e + 5] * mul);
        u.w = pack2<DT>(o[e + 6] * mul, o[e + 7] * mul);
        const int col = c + e, ch = (col % 64) / 8;
        *reinterpret_cast<uint4*>(tile + (col / 64) * (128 * 128) + row * 128 + ((ch ^ (row & 7)) << 4)) = u;
    }
}

// Bits c in [0, 32) with c < n.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

}  // namespace tbe
