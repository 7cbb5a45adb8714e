// The softmax loss's gradients for operands of up to 256 columns (fp32: 128):
// the logits' gradients d never leave the SM.
//
// A CTA holds 128 rows (grad_x) or 128 items (grad_table) in shared memory and
// walks tiles of the others, 128 at a time or, above 128 columns, 64 (shared
// memory holds four of those, but two of 128: the products then waited for
// each tile's fetch, 4150 cycles per 128 of them at 256 columns):
//   grad_x:      S = X W^T,  d = 2^(S c - lse) - [target],           dX += d W
//   grad_table:  S = W X^T,  d likewise, transposed, times g / max,  dW += d X
// (a row's g multiplies its finished grad_x, so rows of any g have all their bits).
// S (fp32) and d (16-bit, the second product's first operand) live in tensor
// memory; the walked tile serves both products, K-major in the first and
// MN-major in the second, so it is fetched once.  That is four products of
// 2 N V D for both gradients where d in memory takes three, but no logit's
// gradient is written or read (6 bytes each, against 4 D operations).
//
// Warp 16 fetches, warp 17 issues the scores' products and warp 18 the sums'
// (one warp's waits for the two left the tensor unit idle: it holds about four
// instructions, a wait takes 100 cycles or more), warps 0 to 15 compute d, eight
// those of the even tiles and eight those of the odd ones: a thread has one line
// of S and half of its columns.  S and d are double buffered beside each other:
// the scores after next are computed as soon as these are read.  fp32's three
// planes of each operand lie in shared memory side by side, d's in tensor memory
// (one d: its products take longer than the next d).
#include "loss_mma.cuh"

namespace tbe {

namespace {

constexpr int kFusedThreads = 608;

template <int DP, int P>
struct Fused {
    static constexpr int BN = loss_fused_walk(DP, P);  // lines of a walked tile
    static constexpr int kFlushTiles = loss_fused_flush(DP, P);
    static constexpr int kHeldPlane = 128 * DP * 2, kTilePlane = BN * DP * 2;
    static constexpr int kHeld = P * kHeldPlane, kTile = P * kTilePlane;
    static constexpr int kStages = P == 3 ? (DP == 64 ? 5 : 2) : DP == 64 ? 6 : DP == 256 ? 4 : 5;
    static constexpr int kStats = 3 * BN * 4;  // bytes of a tile's rows' values
    static constexpr int ring = kHeld, stats = ring + kStages * kTile;
    static constexpr int bytes = stats + kStages * kStats + 1024;
    // tensor memory: two S; two d (16-bit; fp32 one, of three planes); the sums
    // (fp32: of the first planes' products, and 128 columns on of the others)
    static constexpr int d = 2 * BN, kD = P == 3 ? 0 : BN / 2, sums = BN == 128 ? 384 : 256;
    static_assert(d + (P == 3 ? 3 * BN / 2 : BN) <= sums && sums + (P == 3 ? 128 : 0) + DP <= 512, "");
};

struct FusedBars {
    uint64_t held, full[6], empty[6], s_full[2], s_read[2], d_full[2], done[2], last, sums_full, sums_free;
};

// 32 columns of the thread's line: x = S in, d out.
template <int DT, int P, bool ITEMS, int BN>
__device__ __forceinline__ void gradients(float (&x)[32], float c2, float minus_lse, int at, int left,
                                          const float* stats, int line) {
    if constexpr (!ITEMS) {
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
            powers<P>(x[c], x[c + 1], c2, minus_lse, minus_lse);
        }
        if (__any_sync(0xffffffffu, at >= 0 && at < 32)) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
                if (c == at) x[c] -= target_unit<DT>();
        }
        if (left < 32) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
                if (c >= left) x[c] = 0.f;
        }
    } else {
        // columns are rows of x: their values lie in shared memory
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
            const float4 l = *reinterpret_cast<const float4*>(stats + c);
            powers<P>(x[c], x[c + 1], c2, l.x, l.y);
            powers<P>(x[c + 2], x[c + 3], c2, l.z, l.w);
        }
        const int lane = threadIdx.x % 32;
        const int t = __float_as_int(stats[2 * BN + lane]) - (line - lane);  // among the warp's items?
        const uint32_t hit = __ballot_sync(0xffffffffu, t >= 0 && t < 32);
        if (hit) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
                if (hit >> c & 1)
                    if (__float_as_int(stats[2 * BN + c]) == line) x[c] -= target_unit<DT>();
        }
        if (!__all_sync(0xffffffffu, stats[BN + lane] == 1.f)) {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
                const float4 g = *reinterpret_cast<const float4*>(stats + BN + c);
                mul2(x[c], x[c + 1], g.x, g.y);
                mul2(x[c + 2], x[c + 3], g.z, g.w);
            }
        }
    }
}

// fp32's two sums of the thread's line, added (or, `first`, stored) to its row of
// the result, times `unit`, or to a slab as add_slab lays it out.
__device__ __forceinline__ void put_fp32(float* out, float4* part, uint32_t acc, int wide, int group, bool valid, int D,
                                         bool first, float unit) {
    const bool vec = D % 4 == 0 && (uintptr_t)out % 16 == 0;
    for (int c = group * 16; c < wide; c += 64) {
        float x[16], y[16];
        tmem_ld16_pair(acc + c, acc + 128 + c, x, y);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = out ? (x[e] + y[e]) * unit : x[e] + y[e];
        if (!out || vec) {
            float4* to = out ? reinterpret_cast<float4*>(out + c) : part + c / 4 * 128;
            const int step = out ? 1 : 128;
            float4 old[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                old[q] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (!first && (!out || (valid && c + 4 * q < D))) old[q] = to[q * step];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (!out || (valid && c + 4 * q < D))
                    to[q * step] = make_float4(x[4 * q] + old[q].x, x[4 * q + 1] + old[q].y, x[4 * q + 2] + old[q].z,
                                               x[4 * q + 3] + old[q].w);
        } else if (valid) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (c + e < D) out[c + e] = x[e] + (first ? 0.f : out[c + e]);
        }
    }
}

template <int DT, int DP, int P, bool ITEMS>
__device__ __forceinline__ bool fused_body(const LossFused& p, const LossSide& side, const LossFusedMaps& maps, int cta,
                                           unsigned char* smem, FusedBars& bars, uint32_t tmem) {
    using L = Fused<DP, P>;
    constexpr int kStages = L::kStages, BN = L::BN, kFlushTiles = L::kFlushTiles;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // the CTA's tile and the n tiles from `from` on that it walks
    const int tile = cta % side.tiles, slice = cta / side.tiles;
    const int from = (int)((int64_t)side.others * slice / side.slices);
    const int n = (int)((int64_t)side.others * (slice + 1) / side.slices) - from;
    bool ok = true;
    if (n == 0) {  // (a last span of fewer tiles than slices)
    } else if (warp == 16) {
        // ---- loader
        const uint32_t base = smem_u32(smem);
        const int64_t item0 = p.v0 - p.w0;
        auto load = [&](uint32_t dst, const CUtensorMap& map, int64_t row, int boxes, uint64_t* bar) {
#pragma unroll
            for (int plane = 0; plane < P; ++plane)
#pragma unroll
                for (int c = 0; c < DP / 64; ++c)
#pragma unroll
                    for (int r = 0; r < boxes; ++r)
                        load_box(dst + ((plane * (DP / 64) + c) * boxes + r) * kBox, map, c * 64, row + r * 64, plane, bar);
        };
        if (elect_one()) {
            mbar_expect_tx(&bars.held, L::kHeld);
            load(base, ITEMS ? maps.w : maps.x, (ITEMS ? item0 : 0) + (int64_t)tile * 128, 2, &bars.held);
        }
        __syncwarp();
        int i = 0;
        for (; i < n; ++i) {
            const int st = i % kStages;
            if (i >= kStages) ok = mbar_wait_tight(&bars.empty[st], (i / kStages - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (elect_one()) {
                const int64_t other = (int64_t)(from + i) * BN;
                uint64_t* bar = &bars.full[st];
                mbar_expect_tx(bar, L::kTile + (ITEMS ? L::kStats : 0));
                load(base + L::ring + st * L::kTile, ITEMS ? maps.x : maps.w, (ITEMS ? 0 : item0) + other, BN / 64, bar);
                if constexpr (ITEMS) {
                    const float* r = p.rows + other / 128 * kRowValues + other % 128;
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        asm volatile(
                            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
                                "r"(base + L::stats + st * L::kStats + k * BN * 4),
                            "l"(r + k * 128), "r"(BN * 4), "r"(smem_u32(bar))
                            : "memory");
                }
            }
            __syncwarp();
        }
        if (!ok) {  // this CTA's copies in flight land before it ends
            mbar_wait_tight(&bars.held, 0);
            for (int j = tmax(0, i - kStages); j < i; ++j) mbar_wait_tight(&bars.full[j % kStages], (j / kStages) & 1);
        }
    } else if (warp == 17 || warp == 18) {
        // ---- products
        const int ksteps = (p.D + 15) / 16;
        auto wait = [&](uint64_t* bar, int phase) {
            const bool in = mbar_wait_tight(bar, phase & 1);
            const bool all = __all_sync(0xffffffffu, in);
            tcgen05_after_sync();
            return all;
        };
        if (warp == 17) {
            const uint32_t idesc = mma_idesc(DT == DT_BF16, 128, BN);
            const uint64_t held = smem_desc_sw128(smem_u32(smem), 1024);
            const uint64_t walk = smem_desc_sw128(smem_u32(smem) + L::ring, 1024);
            ok = wait(&bars.held, 0);
            for (int i = 0; i < n && ok; ++i) {
                const int st = i % kStages, buf = i & 1;
                ok = (i < 2 || wait(&bars.s_read[buf], i / 2 - 1)) && wait(&bars.full[st], i / kStages);
                if (!ok) break;
                if (elect_one()) {
                    const uint64_t b = walk + (uint64_t)(st * (L::kTile / 16));
#pragma unroll
                    for (int sum = P - 1; sum >= 0; --sum)  // of the planes' numbers: the small products first
#pragma unroll
                        for (int pa = sum; pa >= 0; --pa)
#pragma unroll
                            for (int k = 0; k < DP / 16; ++k)
                                if (k < ksteps)
                                    mma_f16(tmem + buf * BN,
                                            held + pa * (L::kHeldPlane / 16) + (k / 4) * (2 * kBox / 16) + (k % 4) * 2,
                                            b + (sum - pa) * (L::kTilePlane / 16) + (k / 4) * (BN * 128 / 16) + (k % 4) * 2,
                                            idesc, sum + 1 < P || pa < sum || k > 0);
                    mma_commit(&bars.s_full[buf]);
                }
                __syncwarp();
            }
        } else {
            const uint32_t idesc = mma_idesc(DT == DT_BF16, 128, ksteps * 16) | kMnMajorB;
            const uint64_t walk = smem_desc_mn(smem_u32(smem) + L::ring, BN * 128);
            for (int i = 0; i < n && ok; ++i) {
                const int st = i % kStages, buf = i & 1;
                ok = wait(&bars.d_full[buf], i / 2);
                // the sums begin anew every kFlushTiles tiles, once these are in memory
                const bool begins = i % kFlushTiles == 0;
                if (ok && begins && i > 0) ok = wait(&bars.sums_free, i / kFlushTiles - 1);
                if (!ok) break;
                if (elect_one()) {
                    const uint64_t b = walk + (uint64_t)(st * (L::kTile / 16));
#pragma unroll
                    for (int sum = P - 1; sum >= 0; --sum)
#pragma unroll
                        for (int pa = sum; pa >= 0; --pa)
#pragma unroll
                            for (int k = 0; k < BN / 16; ++k)
                                mma_f16_ts(tmem + L::sums + (sum > 0 ? 128 : 0),
                                           tmem + L::d + buf * L::kD + pa * (BN / 2) + k * 8,
                                           b + (sum - pa) * (L::kTilePlane / 16) + k * (2048 / 16), idesc,
                                           !begins || (sum > 0 && (sum + 1 < P || pa < sum)) || k > 0);
                    // (the tile's scores are done with it: d was computed from them)
                    mma_commit(&bars.empty[st]);
                    mma_commit(&bars.done[buf]);
                    if (i + 1 == n)
                        mma_commit(&bars.last);
                    else if (i % kFlushTiles == kFlushTiles - 1)
                        mma_commit(&bars.sums_full);
                }
                __syncwarp();
            }
            // nothing of this CTA arrives on a barrier after its end
            if (ok) ok = wait(&bars.empty[(n - 1) % kStages], (n - 1) / kStages);
        }
    } else {
        // ---- d, then the sums
        const int quarter = warp % 4, group = warp / 4 % 2, buf = warp / 8, line = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        float minus_lse = 0.f;
        int target = -1;
        const float* values = p.rows + (int64_t)tile * kRowValues + line;  // (of the held row)
        if constexpr (!ITEMS) {
            minus_lse = __ldg(values);
            target = __float_as_int(__ldg(values + 256));
        }
        const uint32_t acc = tmem + L::sums + lanes;
        const int wide = (p.D + 15) / 16 * 16;
        const int64_t row = (int64_t)tile * 128 + line;
        int flushed = 0;
        auto put = [&]() {
            const bool first = side.first && flushed == 0;
            const bool valid = row < (ITEMS ? p.v1 - p.v0 : p.N);
            const float times = __ldg(ITEMS ? p.unit : values + 384);
            float4* part = side.part + ((int64_t)slice * side.tiles + tile) * p.cols4 * 128 + line;
            if constexpr (P == 3)
                put_fp32(side.direct ? static_cast<float*>(side.out) + row * p.D : nullptr, part, acc, wide, warp / 4,
                         valid, p.D, first, times);
            else if (side.direct)
                store_rows<DT, 4>(side.out, row * p.D, acc, wide, warp / 4, valid, p.D, p.D % 8 == 0, times);
            else
                add_slab<4, 16>(part, acc, wide, warp / 4, first);
            ++flushed;
        };
        // the first tile's first item of the thread's half (V < 2^31)
        const int item0 = (int)(p.v0 + (int64_t)(from + buf) * BN) + group * (BN / 2);
        int left = (int)p.v1 - item0, at = target - item0, st = buf;
        if (target < 0) at = -1;
        const int mine = (int)(p.v0 + (int64_t)tile * 128) + line;
        int i = buf;
#pragma unroll 1
        while (ok) {  // the tiles of one accumulator, then its way to memory
            const int end = tmin(n, (flushed + 1) * kFlushTiles);
#pragma unroll 1
            for (; i < end; i += 2, left -= 2 * BN, at -= 2 * BN) {
                ok = mbar_wait_tight(&bars.s_full[buf], (i / 2) & 1);
                if (ITEMS && ok) ok = mbar_wait_tight(&bars.full[st], (i / kStages) & 1);  // the rows' values
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tcgen05_after_sync();
                const float* stats = reinterpret_cast<const float*>(smem + L::stats + st * L::kStats) + group * (BN / 2);
                st = st + 2 < kStages ? st + 2 : st + 2 - kStages;
#pragma unroll
                for (int h = 0; h < BN / 2; h += 32) {
                    float x[32];
                    tmem_ld32_issue(tmem + buf * BN + group * (BN / 2) + h + lanes, x);
                    tmem_wait_ld(x, 32);
                    if (h + 32 == BN / 2) {
                        tcgen05_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars.s_read[buf]);
                    }
                    gradients<DT, P, ITEMS, BN>(x, p.c2, minus_lse, at - h, left - h, stats + h, mine);
                    // d's columns are free of the last but one product (fp32: of the last)
                    if (h == 0 && (P == 3 ? i >= 1 : i >= 2)) {
                        ok = P == 3 ? mbar_wait_tight(&bars.done[buf ^ 1], ((i - 1) / 2) & 1)
                                    : mbar_wait_tight(&bars.done[buf], (i / 2 - 1) & 1);
                        ok = __all_sync(0xffffffffu, ok);
                        tcgen05_after_sync();
                    }
#pragma unroll
                    for (int plane = 0; plane < P; ++plane) {
                        uint32_t pk[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            pk[c] = pack2<DT>(x[2 * c], x[2 * c + 1]);
                            if (plane + 1 < P) {
                                x[2 * c] -= __uint_as_float(pk[c] << 16);
                                x[2 * c + 1] -= __uint_as_float(pk[c] & 0xffff0000u);
                            }
                        }
                        tmem_st16(tmem + L::d + buf * L::kD + plane * (BN / 2) + group * (BN / 4) + h / 2 + lanes, pk);
                    }
                }
                if (!ok) break;
                tmem_wait_st();
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.d_full[buf]);
            }
            // (barriers of their own: `done` of the other buffer may be two phases back)
            if (ok) ok = end == n ? mbar_wait_tight(&bars.last, 0) : mbar_wait_tight(&bars.sums_full, flushed & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tcgen05_after_sync();
            put();
            if (end == n) break;
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.sums_free);
        }
    }
    return ok;
}

template <int DT, int DP, int P>
__global__ void __launch_bounds__(kFusedThreads, 1)
    loss_fused_kernel(const LossFused p, const __grid_constant__ LossFusedMaps maps) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ FusedBars bars;
    __shared__ uint32_t slot;
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        mbar_init(&bars.held, 1);
        mbar_init(&bars.last, 1);
        mbar_init(&bars.sums_full, 1);
        mbar_init(&bars.sums_free, 16);
        for (int i = 0; i < Fused<DP, P>::kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.s_read[i], 8);
            mbar_init(&bars.d_full[i], 8);
            mbar_init(&bars.done[i], 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (warp == 17) tmem_alloc(&slot, 512);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = slot;
    chain_wait();
    const int x_ctas = p.x.tiles * p.x.slices, cta = blockIdx.x;
    const bool ok = cta < x_ctas ? fused_body<DT, DP, P, false>(p, p.x, maps, cta, smem, bars, tmem)
                                 : fused_body<DT, DP, P, true>(p, p.w, maps, cta - x_ctas, smem, bars, tmem);
    if (!ok) atomicOr(p.error, ERR_TIMEOUT);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == 17) tmem_dealloc(tmem, 512);
}

template <int OUT>
__global__ void __launch_bounds__(256) loss_finish_kernel(const LossFinish p) {
    chain_wait();
    const int blocks = (p.D + 31) / 32;
    int tile = blockIdx.x / blocks;
    const bool x = tile < p.x.tiles;
    const LossSide& side = x ? p.x : p.w;
    if (!x) tile -= p.x.tiles;
    finish<OUT>(side.part + (int64_t)tile * p.cols4 * 128, (int64_t)side.tiles * p.cols4 * 128, side.slices, side.out,
                (int64_t)tile * 128, (int)tmin<int64_t>(128, (x ? p.x_rows : p.w_rows) - (int64_t)tile * 128), p.D,
                (int)(blockIdx.x % blocks) * 32,
                __ldg(x ? p.rows + (int64_t)tile * kRowValues + 384 + threadIdx.x % 128 : p.unit), threadIdx.x);
}

template <int DT, int DP, int P>
cudaError_t configure() {
    return cudaFuncSetAttribute(loss_fused_kernel<DT, DP, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Fused<DP, P>::bytes);
}

template <int DT, int DP, int P = 1>
cudaError_t launch(const LossFused& p, const LossFusedMaps& maps, cudaStream_t s) {
    const int grid = p.x.tiles * p.x.slices + p.w.tiles * p.w.slices;
    return launch_chained_smem(loss_fused_kernel<DT, DP, P>, dim3(grid), dim3(kFusedThreads), Fused<DP, P>::bytes, s, p,
                               maps);
}

template <int DT>
cudaError_t launch_width(const LossFused& p, const LossFusedMaps& maps, cudaStream_t s) {
    if (p.D <= 64) return launch<DT, 64>(p, maps, s);
    if (p.D <= 128) return launch<DT, 128>(p, maps, s);
    if (p.D <= 192) return launch<DT, 192>(p, maps, s);
    return launch<DT, 256>(p, maps, s);
}

}  // namespace

cudaError_t loss_fused_configure() {
    cudaError_t e = configure<DT_F16, 64, 1>();
    if (e == cudaSuccess) e = configure<DT_F16, 128, 1>();
    if (e == cudaSuccess) e = configure<DT_F16, 192, 1>();
    if (e == cudaSuccess) e = configure<DT_F16, 256, 1>();
    if (e == cudaSuccess) e = configure<DT_BF16, 64, 1>();
    if (e == cudaSuccess) e = configure<DT_BF16, 128, 1>();
    if (e == cudaSuccess) e = configure<DT_BF16, 192, 1>();
    if (e == cudaSuccess) e = configure<DT_BF16, 256, 1>();
    if (e == cudaSuccess) e = configure<DT_BF16, 64, 3>();
    if (e == cudaSuccess) e = configure<DT_BF16, 128, 3>();
    return e;
}

cudaError_t launch_loss_fused(const LossFused& p, const LossFusedMaps& maps, int dtype, cudaStream_t s) {
    if (dtype == DT_F32) return p.D <= 64 ? launch<DT_BF16, 64, 3>(p, maps, s) : launch<DT_BF16, 128, 3>(p, maps, s);
    return dtype == DT_F16 ? launch_width<DT_F16>(p, maps, s) : launch_width<DT_BF16>(p, maps, s);
}

cudaError_t launch_loss_finish(const LossFinish& p, int dtype, cudaStream_t s) {
    const dim3 grid((unsigned)(p.x.tiles + p.w.tiles) * ((p.D + 31) / 32));
    return dtype == DT_F32   ? launch_chained(loss_finish_kernel<DT_F32>, grid, dim3(256), s, p)
           : dtype == DT_F16 ? launch_chained(loss_finish_kernel<DT_F16>, grid, dim3(256), s, p)
                             : launch_chained(loss_finish_kernel<DT_BF16>, grid, dim3(256), s, p);
}

}  // namespace tbe
