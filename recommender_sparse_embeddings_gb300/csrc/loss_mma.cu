// The softmax loss's forward kernel and the backward pass's for wide operands, on
// the tensor cores; see loss_mma.cuh.
#include "loss_mma.cuh"

namespace tbe {

namespace {

constexpr int kForwardThreads = 576;
constexpr float kLargeSum = 8192.f;

struct LossBars {
    uint64_t full[kLossStages], empty[kLossStages], a_full[2], a_empty[2], acc_full[2], acc_empty[2];
};

__device__ __forceinline__ void store_box(const CUtensorMap& map, uint32_t src, int col, int row, int plane) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(&map),
                 "r"(col), "r"(row), "r"(plane), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ void store_read_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// A tile of products: `steps` of 64 along the sum, `wide` columns.
struct Product {
    int kind;
    int row0;         // rows of A's tile: X rows, d rows, items of the piece
    int64_t col0;     // of B's tile: first item (scores) or first column (gx, gw)
    int k0, kblocks;  // along the sum, blocks of 64
    int wide;
    int slab;
    int last_steps;  // scores: steps of 16 columns in the last block
    bool begins;     // a sum's first part
};

__device__ __forceinline__ int columns_of(int64_t left) { return (int)tmin<int64_t>(256, (left + 15) / 16 * 16); }

__device__ __forceinline__ Product score_tile(int64_t V, int D, int row0, int64_t item) {
    return Product{ITEM_D, row0, item, 0, (D + 63) / 64, columns_of(V - item), 0, ((D - 1) % 64 + 16) / 16, true};
}

// Its first part, or the one after t, of `part` blocks; `rest` are still to come then.
__device__ __forceinline__ void score_part(Product& t, int D, int part, bool first, int& rest) {
    t.k0 = first ? 0 : t.k0 + t.kblocks;
    if (first) rest = (D + 63) / 64;
    t.kblocks = tmin(rest, part);
    rest -= t.kblocks;
    t.last_steps = rest > 0 ? 4 : ((D - 1) % 64 + 16) / 16;
}

// Work item i of a backward launch: the long ones first.
__device__ __forceinline__ Product step_item(const LossStep& p, int i) {
    Product t{};
    t.begins = true;
    if (i < p.n_gw) {
        const int tiles = (p.p_items + 127) / 128, blocks = (int)((p.N + 63) / 64);
        const int tile = i % tiles, rest = i / tiles, ct = rest % p.col_tiles;
        t.kind = ITEM_GW;
        t.slab = rest / p.col_tiles;
        t.row0 = tile * 128;
        t.col0 = ct * 256;
        t.k0 = (int)((int64_t)blocks * t.slab / p.w_slabs);
        t.kblocks = (int)((int64_t)blocks * (t.slab + 1) / p.w_slabs) - t.k0;
        t.wide = columns_of(p.D - t.col0);
        return t;
    }
    i -= p.n_gw;
    if (i < p.n_gx) {
        const int blocks = (p.p_items + 63) / 64;
        const int tile = i % p.row_tiles, rest = i / p.row_tiles, ct = rest % p.col_tiles;
        t.kind = ITEM_GX;
        t.slab = rest / p.col_tiles;
        t.row0 = tile * 128;
        t.col0 = ct * 256;
        t.k0 = (int)((int64_t)blocks * t.slab / p.x_slabs);
        t.kblocks = (int)((int64_t)blocks * (t.slab + 1) / p.x_slabs) - t.k0;
        t.wide = columns_of(p.D - t.col0);
        return t;
    }
    i -= p.n_gx;
    if (i < p.n_d) return score_tile(p.V, p.D, i % p.row_tiles * 128, p.d0 + (int64_t)(i / p.row_tiles) * 256);
    i -= p.n_d;
    t.kind = i < p.n_fin_w ? ITEM_FIN_W : ITEM_FIN_X;
    if (i >= p.n_fin_w) i -= p.n_fin_w;
    const int blocks = (p.D + 31) / 32;
    t.row0 = i / blocks * 128;
    t.col0 = i % blocks * 32;
    return t;
}

// The operands' way through shared memory.  One plane: stages of a tile of A (2
// boxes) and of B (4).  fp32's three: A's planes of a block stay for the block's
// six products, twice 3 tiles; B's planes pass in three stages, each meeting the
// planes of A that matter beside it; the first planes come once more for the
// large products.  That is 192 KB for what 288 KB of single products would be (the
// L2 cache's reads bound fp32's passes).
template <int P>
struct Ring {
    static constexpr int kStages = P == 3 ? 3 : 4;
    static constexpr int kStage = P == 3 ? 4 * kBox : 6 * kBox;
    static constexpr int b = P == 3 ? 2 * 3 * 2 * kBox : 2 * kBox;  // of the first stage
};
static_assert(Ring<3>::b + Ring<3>::kStages * Ring<3>::kStage <= kLossStages * kStageBytes, "");

// fp32's passes over a sum: the small products, then the large; both at once
// where the sum is one block.
enum : int { kSmall = 0, kLarge = 1, kBoth = 2 };
template <int P>
__device__ __forceinline__ int first_pass(const Product& t) {
    return P == 1 ? kLarge : t.kblocks == 1 ? kBoth : kSmall;
}
template <int P>
__device__ __forceinline__ int last_pass(const Product& t) {
    return P == 3 && t.kblocks == 1 ? kBoth : kLarge;
}

template <int P, typename Next>
__device__ bool produce(unsigned char* smem, LossBars& bars, const LossMaps& maps, int64_t w0, int64_t p_row, Next next) {
    using R = Ring<P>;
    int n = 0, blocks = 0;  // stages and (P = 3) blocks so far
    bool ok = true;
    Product t;
    const uint32_t base = smem_u32(smem);
    while (ok && next(t)) {
        if (t.kind >= ITEM_FIN_W) continue;
        const int slabs = (t.wide + 63) / 64;
        auto load_a = [&](uint32_t a, int k, int plane, uint64_t* bar) {
            if (t.kind == ITEM_D) {
                load_box(a, maps.x, k, t.row0, plane, bar);
                load_box(a + kBox, maps.x, k, t.row0 + 64, plane, bar);
            } else if (t.kind == ITEM_GX) {
                load_box(a, maps.d_in, k, t.row0, plane, bar);
                load_box(a + kBox, maps.d_in, k, t.row0 + 64, plane, bar);
            } else {
                load_box(a, maps.d_in, t.row0, k, plane, bar);
                load_box(a + kBox, maps.d_in, t.row0 + 64, k, plane, bar);
            }
        };
        auto load_b = [&](uint32_t b, int k, int plane, uint64_t* bar) {
            for (int j = 0; j < slabs; ++j)
                if (t.kind == ITEM_D)
                    load_box(b + j * kBox, maps.w, k, t.col0 - w0 + j * 64, plane, bar);
                else if (t.kind == ITEM_GX)
                    load_box(b + j * kBox, maps.pw, (int)t.col0 + j * 64, p_row + k, plane, bar);
                else
                    load_box(b + j * kBox, maps.x, (int)t.col0 + j * 64, k, plane, bar);
        };
        for (int pass = first_pass<P>(t); pass <= last_pass<P>(t) && ok; ++pass)
            for (int s = 0; s < t.kblocks && ok; ++s) {
                const int k = (t.k0 + s) * 64;
                if constexpr (P == 3) {
                    const int ab = blocks & 1;
                    if (blocks >= 2) ok = mbar_wait_tight(&bars.a_empty[ab], (blocks / 2 - 1) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (elect_one()) {
                        const int planes = pass == kLarge ? 1 : 3;
                        mbar_expect_tx(&bars.a_full[ab], planes * 2 * kBox);
                        for (int plane = 0; plane < planes; ++plane)
                            load_a(base + (ab * 3 + plane) * 2 * kBox, k, plane, &bars.a_full[ab]);
                    }
                    __syncwarp();
                    ++blocks;
                }
                for (int plane = pass == kLarge ? 0 : 2; plane >= 0 && ok; --plane, ++n) {
                    const int st = n % R::kStages;
                    if (n >= R::kStages) ok = mbar_wait_tight(&bars.empty[st], (n / R::kStages - 1) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_expect_tx(&bars.full[st], ((P == 3 ? 0 : 2) + slabs) * kBox);
                        if constexpr (P == 1) load_a(base + st * R::kStage, k, 0, &bars.full[st]);
                        load_b(base + R::b + st * R::kStage, k, plane, &bars.full[st]);
                    }
                    __syncwarp();
                }
            }
    }
    // where a wait ran out: this CTA's copies in flight land before it ends
    if (!ok) {
        for (int i = tmax(0, n - R::kStages); i < n; ++i)
            mbar_wait_tight(&bars.full[i % R::kStages], (i / R::kStages) & 1);
        for (int i = tmax(0, blocks - 2); i < blocks; ++i) mbar_wait_tight(&bars.a_full[i & 1], (i / 2) & 1);
    }
    return ok;
}

template <int DT, int P, typename Next>
__device__ bool multiply(unsigned char* smem, LossBars& bars, uint32_t tmem, Next next) {
    using R = Ring<P>;
    int n = 0, blocks = 0, tile = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
        const bool in = mbar_wait_tight(bar, parity & 1);
        const bool all = __all_sync(0xffffffffu, in);
        tcgen05_after_sync();
        return all;
    };
    const uint32_t base = smem_u32(smem);
    Product t;
    while (ok && next(t)) {
        if (t.kind >= ITEM_FIN_W) continue;
        const int buf = tile & 1;
        if (tile >= 2) ok = wait(&bars.acc_empty[buf], tile / 2 - 1);
        const bool a_mn = t.kind == ITEM_GW, b_mn = t.kind != ITEM_D;
        const uint32_t idesc =
            mma_idesc(DT == DT_BF16, 128, t.wide) | (a_mn ? 1u << 15 : 0u) | (b_mn ? kMnMajorB : 0u);
        const uint64_t da = a_mn ? smem_desc_mn(base, kBox) : smem_desc_sw128(base, 1024);
        const uint64_t db = b_mn ? smem_desc_mn(base + R::b, kBox) : smem_desc_sw128(base + R::b, 1024);
        const int ka = a_mn ? 2048 / 16 : 2, kb = b_mn ? 2048 / 16 : 2;
        for (int pass = first_pass<P>(t); pass <= last_pass<P>(t) && ok; ++pass)
            for (int s = 0; s < t.kblocks && ok; ++s) {
                const int steps = t.kind == ITEM_D && s + 1 == t.kblocks ? t.last_steps : 4;  // of 16 along the sum
                const int ab = blocks & 1;
                if constexpr (P == 3) {
                    ok = wait(&bars.a_full[ab], blocks / 2);
                    ++blocks;
                }
                for (int plane = pass == kLarge ? 0 : 2; plane >= 0 && ok; --plane, ++n) {
                    const int st = n % R::kStages;
                    ok = wait(&bars.full[st], n / R::kStages);
                    if (!ok) break;
                    if (elect_one()) {
                        const uint64_t b = db + (uint64_t)(st * (R::kStage / 16));
                        // A's planes that matter beside this one of B; the first ones' product comes last
                        for (int pa = pass == kLarge ? 0 : 2 - plane; pa >= (pass == kSmall && plane == 0 ? 1 : 0); --pa) {
                            const uint64_t a =
                                da + (uint64_t)(P == 3 ? (ab * 3 + pa) * (2 * kBox / 16) : st * (R::kStage / 16));
                            const bool begins = s == 0 && (P == 1 || (pass != kLarge && plane == 2));
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (k < steps) mma_f16(tmem + buf * 256, a + k * ka, b + k * kb, idesc, !begins || k > 0);
                        }
                        mma_commit(&bars.empty[st]);
                        if (plane == 0) {
                            if constexpr (P == 3) mma_commit(&bars.a_empty[ab]);
                            if (pass != kSmall && s + 1 == t.kblocks) mma_commit(&bars.acc_full[buf]);
                        }
                    }
                    __syncwarp();
                }
            }
        ++tile;
    }
    // nothing of this CTA arrives on a barrier after its end
    if (ok && n > 0) ok = wait(&bars.empty[(n - 1) % R::kStages], (n - 1) / R::kStages);
    if (P == 3 && ok && blocks > 0) ok = wait(&bars.a_empty[(blocks - 1) & 1], (blocks - 1) / 2);
    return ok;
}

// N columns of the thread's line of a part of the scores, added to x or stored there.
template <bool ADD, int N>
__device__ __forceinline__ void take_scores(float (&x)[N], uint32_t acc) {
#pragma unroll
    for (int c = 0; c < N; c += 16) {
        float y[16];
        tmem_ld16(acc + c, y);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[c + e] = ADD ? x[c + e] + y[e] : y[e];
    }
}

// 32 columns of one row in staging: the warp's tile of 32 rows x 128 bytes in
// the 128-byte swizzle.
__device__ __forceinline__ void stage_row(unsigned char* staging, int lane, int half, const uint32_t* pk) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(staging + lane * 128 + (((half * 4 + c) ^ (lane & 7)) << 4)) =
            make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
}

// d of the warp's 32 rows and one of its two slabs of 64 items.
template <int DT, int P>
__device__ __forceinline__ void d_slab(float* x, float minus_lse, float coef, int target, float c2, int64_t item0, int64_t V,
                                       unsigned char* staging, const CUtensorMap& map, int col, int row, int64_t rows,
                                       int lane) {
#pragma unroll
    for (int c = 0; c < 64; c += 2) {
        powers<P>(x[c], x[c + 1], c2, minus_lse, minus_lse);
    }
    const int at = (int)tmin<int64_t>(tmax<int64_t>(target - item0, -1), 64);  // (target -1: before any item)
    if (__any_sync(0xffffffffu, at >= 0 && at < 64)) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
            if (c == at) x[c] -= target_unit<DT>();
    }
    const int64_t left = V - item0;
    if (left < 64) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
            if (c >= left) x[c] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < 64; c += 2) mul2(x[c], x[c + 1], coef, coef);
#pragma unroll
    for (int plane = 0; plane < P; ++plane) {
        if (lane == 0) store_read_wait();
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                pk[c] = pack2<DT>(x[32 * h + 2 * c], x[32 * h + 2 * c + 1]);
                if constexpr (P == 3) {
                    x[32 * h + 2 * c] -= bf16_bits_to_float(pk[c] & 0xffffu);
                    x[32 * h + 2 * c + 1] -= __uint_as_float(pk[c] & 0xffff0000u);
                }
            }
            stage_row(staging, lane, h, pk);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row < rows) store_box(map, smem_u32(staging), col, row, plane);
    }
}

template <int WARP, int READERS>  // the warp that allocates; warps that read an accumulator
__device__ __forceinline__ uint32_t begin(LossBars& bars, uint32_t* slot) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < kLossStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.a_full[i], 1);
            mbar_init(&bars.a_empty[i], 1);
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], READERS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (threadIdx.x / 32 == WARP) tmem_alloc(slot, 512);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    return *slot;
}

template <int WARP>
__device__ __forceinline__ void end(uint32_t tmem, bool ok, uint32_t* error) {
    if (!ok) atomicOr(error, ERR_TIMEOUT);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (threadIdx.x / 32 == WARP) tmem_dealloc(tmem, 512);
}

// Backward pass: one launch's work items.  PARTS (fp32, above 512 columns): a tile of
// scores has several accumulators.
template <int DT, int P, bool PARTS = false>
__global__ void __launch_bounds__(kLossThreads, 1)
    loss_step_kernel(const LossStep p, const __grid_constant__ LossMaps maps) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ LossBars bars;
    __shared__ uint32_t slot;
    const uint32_t tmem = begin<9, 8>(bars, &slot);
    chain_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // the products in turn (the long items first), then this CTA's share of d,
    // the results in turn
    const int products = p.n_gw + p.n_gx, results = products + p.n_d, n_items = results + p.n_fin_w + p.n_fin_x;
    int a = blockIdx.x, b = products + p.d_from[blockIdx.x], f = results + blockIdx.x;
    const int b_end = products + p.d_from[blockIdx.x + 1];
    // blocks of the item that are still to come: its sum goes to memory in parts (with
    // 16-bit types a sum that goes to the result at once is short enough)
    constexpr int kPart = P == 3 ? kFlush : kLongSum / 64;
    const int part = PARTS ? score_part_blocks(p.D) : 0;
    int rest = 0;
    auto next = [&](Product& t) {
        for (;;) {
            int i;
            if (PARTS && rest > 0 && t.kind == ITEM_D) {
                score_part(t, p.D, part, false, rest);
                return true;
            }
            if (rest > 0) {
                t.k0 += t.kblocks;
                t.kblocks = tmin(rest, kPart);
                t.begins = false;
                rest -= t.kblocks;
                return true;
            }
            if (a < products) {
                i = a;
                a += gridDim.x;
            } else if (b < b_end) {
                i = b++;
            } else if (f < n_items) {
                i = f;
                f += gridDim.x;
            } else {
                return false;
            }
            t = step_item(p, i);
            if (PARTS && t.kind == ITEM_D) score_part(t, p.D, part, true, rest);
            if (t.kind > ITEM_GX) return true;
            if (t.kblocks == 0) continue;  // (the last piece has fewer blocks than slabs)
            rest = tmax(0, t.kblocks - kPart);
            t.kblocks -= rest;
            return true;
        }
    };
    bool ok = true;
    if (warp == 8) {
        ok = produce<P>(smem, bars, maps, p.dw0, p.p0 - p.pw0, next);
    } else if (warp == 9) {
        ok = multiply<DT, P>(smem, bars, tmem, next);
    } else {
        constexpr int OUT = P == 3 ? DT_F32 : DT;
        unsigned char* staging = smem + kLossStages * kStageBytes + warp * kStagingBytes;
        const int quarter = warp % 4, group = warp / 4;
        const float unit = __ldg(p.unit);
        int tile = 0;
        Product t;
        while (next(t)) {
            if (t.kind >= ITEM_FIN_W) {
                const bool w = t.kind == ITEM_FIN_W;
                const int tiles = w ? (p.f_items + 127) / 128 : p.row_tiles;
                finish<OUT>((w ? p.f_part : p.x_part) + (int64_t)(t.row0 / 128) * p.cols4 * 128,
                            (int64_t)tiles * p.cols4 * 128, w ? p.w_slabs : p.x_slabs, w ? p.gw : p.gx,
                            (w ? p.f0 : 0) + t.row0, (int)tmin<int64_t>(128, (w ? p.f_items : p.N) - t.row0), p.D,
                            (int)t.col0, unit, threadIdx.x);
                continue;
            }
            const int buf = tile & 1;
            float minus_lse = 0.f, coef = 0.f;
            int target = -1;
            if (t.kind == ITEM_D) {
                const float* r = p.rows + (int64_t)(t.row0 / 128) * kRowValues + quarter * 32 + lane;
                minus_lse = __ldg(r);
                coef = __ldg(r + 128);
                target = __float_as_int(__ldg(r + 256));
            }
            if (ok) ok = mbar_wait_tight(&bars.acc_full[buf], (tile / 2) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tcgen05_after_sync();
            const uint32_t acc = tmem + buf * 256 + ((uint32_t)(quarter * 32) << 16);
            auto release = [&]() {
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.acc_empty[tile & 1]);
                ++tile;
            };
            if (PARTS && t.kind == ITEM_D) {
                float x[128];
                take_scores<false>(x, acc + group * 128);
                release();
                while (rest > 0) {
                    next(t);
                    ok = mbar_wait_tight(&bars.acc_full[tile & 1], (tile / 2) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tcgen05_after_sync();
                    take_scores<true>(x, tmem + (tile & 1) * 256 + ((uint32_t)(quarter * 32) << 16) + group * 128);
                    release();
                }
                if (!ok) break;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int c = group * 128 + s * 64;
                    if (t.col0 + c >= p.V) break;
                    d_slab<DT, P>(x + s * 64, minus_lse, coef, target, p.c2, t.col0 + c, p.V, staging, maps.d_out,
                                  (int)(t.col0 - p.d0) + c, t.row0 + quarter * 32, p.N, lane);
                }
                continue;
            }
            if (t.kind == ITEM_D) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int c = group * 128 + s * 64;
                    if (t.col0 + c >= p.V) break;
                    float x[64];
                    tmem_ld32_issue(acc + c, x);
                    tmem_ld32_issue(acc + c + 32, x + 32);
                    tmem_wait_ld(x, 64);
                    d_slab<DT, P>(x, minus_lse, coef, target, p.c2, t.col0 + c, p.V, staging, maps.d_out, (int)(t.col0 - p.d0) + c,
                                  t.row0 + quarter * 32, p.N, lane);
                }
            } else if (t.kind == ITEM_GW && p.w_slabs == 1) {
                const int r = t.row0 + quarter * 32 + lane;
                store_rows<OUT, 2>(p.gw, (p.p0 + r) * p.D + t.col0, acc, t.wide, group, r < p.p_items,
                                (int)(p.D - t.col0), p.D % 8 == 0, unit, !t.begins);
            } else {
                const int tiles = t.kind == ITEM_GX ? p.row_tiles : (p.p_items + 127) / 128;
                float4* to = (t.kind == ITEM_GX ? p.x_part : p.w_part) +
                             ((int64_t)t.slab * tiles + t.row0 / 128) * p.cols4 * 128 + t.col0 / 4 * 128 +
                             quarter * 32 + lane;
                add_slab<2>(to, acc, t.wide, group, t.begins && (t.kind == ITEM_GW || p.first));
            }
            release();
        }
        if (lane == 0) store_wait();
    }
    end<9>(tmem, ok, p.error);
}

// Forward pass: a CTA's item is a tile of 128 rows and a slice of the table,
// whose maximum and sum its threads (a row and a quarter of a tile's columns
// each) carry in registers.  The maximum moves only when 32 terms' sum against the
// last one exceeds 2^13 (below, an fp32 sum loses nothing by it); otherwise no
// maximum is looked for (a third of the loop's instructions).
// PARTS: above 512 columns, a tile has several accumulators.
template <int DT, int P, bool PARTS>
__global__ void __launch_bounds__(kForwardThreads, 1)
    loss_forward_kernel(const LossForward p, const __grid_constant__ LossMaps maps) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ LossBars bars;
    __shared__ uint32_t slot;
    const uint32_t tmem = begin<17, 16>(bars, &slot);
    chain_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int n_items = p.row_tiles * p.slices;
    const int part = PARTS ? score_part_blocks(p.D) : 0;
    int item = blockIdx.x, tiles = 0, rest = 0;  // tiles: left of the item, rest: blocks of the tile
    // (called with the same t: all but an item's first tile only move it on)
    auto next = [&](Product& t) {
        if (PARTS && rest > 0) {
            score_part(t, p.D, part, false, rest);
            return true;
        }
        while (tiles == 0) {
            if (item >= n_items) return false;
            const int slice = item / p.row_tiles;
            const int at = (int)((int64_t)p.item_tiles * slice / p.slices);
            tiles = (int)((int64_t)p.item_tiles * (slice + 1) / p.slices) - at;  // (none: a short last span's)
            t = score_tile(p.v1, p.D, item % p.row_tiles * 128, p.v0 + (int64_t)(at - 1) * 256);
            t.slab = slice;
            item += gridDim.x;
        }
        t.col0 += 256;
        t.wide = --tiles == 0 ? columns_of(p.v1 - t.col0) : 256;
        if (PARTS) score_part(t, p.D, part, true, rest);
        return true;
    };
    bool ok = true;
    if (warp == 16) {
        ok = produce<P>(smem, bars, maps, p.w0, 0, next);
    } else if (warp == 17) {
        ok = multiply<DT, P>(smem, bars, tmem, next);
    } else {
        // (an item's tiles in a loop of its own: `next` for each of them took as
        // long as their arithmetic)
        const int quarter = warp % 4, group = warp / 4;
        int tile = 0;
        Product t;
        while (ok && next(t)) {
            const int count = tiles + 1;
            tiles = rest = 0;
            const int64_t row = t.row0 + quarter * 32 + lane;
            float m = -INFINITY, l = 0.f, picked = 0.f;
            int left = (int)(p.v1 - t.col0) - group * 64;  // items from the quarter on
            int mine = -1;                                 // the target's place among them (V < 2^31)
            bool found = false;
            if (row < p.N) {
                if (!p.first) {
                    const float2 y = p.part[(row * p.slices + t.slab) * 4 + group];
                    m = y.x;
                    l = y.y;
                }
                const int64_t target = p.index64 ? static_cast<const int64_t*>(p.targets)[row]
                                                 : static_cast<const int32_t*>(p.targets)[row];
                if (target >= p.V)
                    atomicOr(p.error, ERR_OOB);
                else if (target >= 0)
                    mine = (int)(target - t.col0) - group * 64;
            }
            const uint32_t acc0 = tmem + group * 64 + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
            for (int j = 0; j < count; ++j, ++tile, left -= 256, mine -= 256) {
                auto arrived = [&]() {
                    ok = mbar_wait_tight(&bars.acc_full[tile & 1], (tile / 2) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    tcgen05_after_sync();
                    return ok;
                };
                auto release = [&]() {
                    tcgen05_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.acc_empty[tile & 1]);
                };
                const bool picks = __any_sync(0xffffffffu, mine >= 0 && mine < 64);
                // 32 columns from c on
                auto take = [&](float (&x)[32], int c) {
                    if (picks && __any_sync(0xffffffffu, mine >= c && mine < c + 32)) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)  // (in C++ it becomes an indexed copy in local memory)
                            asm volatile("{\n\t.reg .pred q;\n\tsetp.eq.s32 q, %1, 0;\n\t@q mov.f32 %0, %2;\n\t}"
                                         : "+f"(picked)
                                         : "r"(mine - c - e), "f"(x[e]));
                        found |= mine >= c && mine < c + 32;
                    }
                    auto sum = [&]() {
                        float s0 = 0.f, s1 = 0.f;
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float y0 = x[e], y1 = x[e + 1];
                            powers<P>(y0, y1, p.c2, -m, -m);
                            add2(s0, s1, y0, y1);
                        }
                        return s0 + s1;
                    };
                    float s = sum();
                    if (__any_sync(0xffffffffu, !(s <= kLargeSum))) {  // (m = -inf, at first, too)
                        float u[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) u[e] = fmaxf(max3(x[e], x[e + 8], x[e + 16]), x[e + 24]);
                        const float top = fmaxf(max3(max3(u[0], u[1], u[2]), u[3], u[4]), max3(u[5], u[6], u[7])) * p.c2;
                        // (only where it is the row's own: a neighbour's logits change no bits)
                        const float to = s <= kLargeSum ? m : fmaxf(m, top);
                        l *= ex2(P == 3 ? (m - to) * kLog2e : m - to);  // (m = -inf: 0)
                        m = to;
                        s = sum();
                    }
                    l += s;
                };
                if constexpr (PARTS) {
                    float x[32], y[32];
                    if (!arrived()) break;
                    take_scores<false>(x, acc0 + (tile & 1) * 256);
                    take_scores<false>(y, acc0 + (tile & 1) * 256 + 32);
#pragma unroll 1
                    for (int k = part; k < (p.D + 63) / 64; k += part) {
                        release();
                        ++tile;
                        if (!arrived()) break;
                        take_scores<true>(x, acc0 + (tile & 1) * 256);
                        take_scores<true>(y, acc0 + (tile & 1) * 256 + 32);
                    }
                    if (!ok) break;
                    release();
                    if (left < 64) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            if (e >= left) x[e] = -INFINITY;
                            if (e + 32 >= left) y[e] = -INFINITY;
                        }
                    }
                    if (left > 0) take(x, 0);
                    if (left > 32) take(y, 32);
                    continue;
                }
                if (!arrived()) break;
                const uint32_t acc = acc0 + (tile & 1) * 256;
                if (left >= 64) {
                    float x[32], y[32];
                    tmem_ld32_issue(acc, x);
                    tmem_wait_ld(x, 32);
                    tmem_ld32_issue(acc + 32, y);
                    take(x, 0);
                    tmem_wait_ld(y, 32);
                    release();
                    take(y, 32);
                } else {
#pragma unroll 1
                    for (int c = 0; c < left; c += 32) {
                        float x[32];
                        tmem_ld32_issue(acc + c, x);
                        tmem_wait_ld(x, 32);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (e >= left - c) x[e] = -INFINITY;
                        take(x, c);
                    }
                    release();
                }
            }
            if (ok && row < p.N) {
                p.part[(row * p.slices + t.slab) * 4 + group] = make_float2(m, l);
                if (found) p.picked[row] = picked * p.c2;
            }
        }
    }
    end<17>(tmem, ok, p.error);
}

template <int DT, int P>
cudaError_t configure() {
    cudaError_t e = cudaFuncSetAttribute(loss_step_kernel<DT, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLossSmem);
    if (e == cudaSuccess && P == 3)
        e = cudaFuncSetAttribute(loss_step_kernel<DT, P, P == 3>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLossSmem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(loss_forward_kernel<DT, P, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLossSmem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(loss_forward_kernel<DT, P, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLossSmem);
    return e;
}

}  // namespace

cudaError_t loss_mma_configure() {
    cudaError_t e = configure<DT_F16, 1>();
    if (e == cudaSuccess) e = configure<DT_BF16, 1>();
    if (e == cudaSuccess) e = configure<DT_BF16, 3>();
    return e;
}

template <bool PARTS>
static cudaError_t launch_forward(const LossForward& p, const LossMaps& maps, int dtype, int grid, cudaStream_t s) {
    auto* kernel = dtype == DT_F32   ? loss_forward_kernel<DT_BF16, 3, PARTS>
                   : dtype == DT_F16 ? loss_forward_kernel<DT_F16, 1, PARTS>
                                     : loss_forward_kernel<DT_BF16, 1, PARTS>;
    return launch_chained_smem(kernel, dim3(grid), dim3(kForwardThreads), kLossSmem, s, p, maps);
}

cudaError_t launch_loss_forward(const LossForward& p, const LossMaps& maps, int dtype, int grid, cudaStream_t s) {
    return p.D > kScorePart * 64 ? launch_forward<true>(p, maps, dtype, grid, s)
                                 : launch_forward<false>(p, maps, dtype, grid, s);
}

cudaError_t launch_loss_step(const LossStep& p, const LossMaps& maps, int dtype, int grid, cudaStream_t s) {
    auto* kernel = dtype == DT_F16          ? loss_step_kernel<DT_F16, 1>
                   : dtype == DT_BF16       ? loss_step_kernel<DT_BF16, 1>
                   : p.D <= kScorePart * 64 ? loss_step_kernel<DT_BF16, 3>
                                            : loss_step_kernel<DT_BF16, 3, true>;
    return launch_chained_smem(kernel, dim3(grid), dim3(kLossThreads), kLossSmem, s, p, maps);
}

}  // namespace tbe
