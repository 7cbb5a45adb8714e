// Tensor-core building blocks of the attention kernels: tiles of 16-bit rows
// in shared memory, operands in tensor memory, and bounded waits.
//
// Tiles.  A tile of R rows (tokens) of DP columns is stored as DP / 64 slabs
// of R rows x 128 bytes in the 128-byte swizzle: 16-byte chunk c of row r at
// chunk c ^ (r & 7).  One copy serves as a K-major operand (the product runs
// over the columns: Q K^T) and as an MN-major one (over the rows: P V), by
// its descriptor alone, so nothing is transposed.
#pragma once

#include "attention.cuh"
#include "tcgen05.cuh"

namespace tbe {

// Bounded wait without a sleep between the tries: each try may suspend the
// thread up to the hint (about 2 us), so 2^20 tries end within seconds.
__device__ __forceinline__ bool mbar_wait_tight(uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    for (int i = 0; i < kSpinLimit; ++i) {
        uint32_t ok;
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

// Descriptor of an MN-major operand in the tile layout: 8-row groups (along
// K) are 1024 bytes apart, 64-column blocks (along M or N) one slab.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr, uint32_t slab) {
    return smem_desc(addr, slab, 1024u) | ((uint64_t)2u << 61);
}

// Bits of the instruction descriptor that make A or B MN-major.
constexpr uint32_t kMnMajorA = 1u << 15;
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

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]),
        "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
        "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(taddr)
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
    const int n = real ? 16 : 0;  // 0: sixteen zero bytes, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows [from, from + COUNT) of a tile of ROWS rows whose row 0 is row `row0`
// of a history (zeros from row `len` on and from column D on), by one warp.
// 16-bit elements.
template <int ROWS, int DP, int COUNT = ROWS>
__device__ __forceinline__ void load_tile_async(uint32_t dst, const Rows& r, int64_t token0, int head, int row0,
                                                int len, int D, int lane, int from = 0) {
    const int chunk = lane % 8;
    const uint16_t* base = static_cast<const uint16_t*>(r.data) + head * r.head_stride + chunk * 8;
    const uint16_t* src = base + (token0 + row0) * r.token_stride;
#pragma unroll
    for (int slab = 0; slab < DP / 64; ++slab) {
        const int col = slab * 64 + chunk * 8;
        const bool inside = col < D;
        for (int row = from + lane / 8; row < from + COUNT; row += 4) {
            const bool real = inside && row0 + row < len;
            const uint16_t* p = real ? src + row * r.token_stride + slab * 64 : base;
            cp_async16(dst + slab * (ROWS * 128) + row * 128 + ((chunk ^ (row & 7)) << 4), p, real);
        }
    }
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
