// Attention over ragged histories on the tensor cores (tcgen05), backward.
//
// Two kernels, each summing its gradients inside one CTA in a fixed order
// (no atomics, no fp32 copies of the gradients in memory), at the price of
// computing the logits and their gradients twice (eight products, not five):
//
// dq (128 queries of one head; key blocks of 64):
//   S = Q K^T, dP = G V^T, dS = P (dP - delta), dQ += dS K, R += P K
// dkv (128 keys of one key-value head; query blocks of 64, over the group's
// heads), transposed so that P^T and dS^T are products' first operands and
// stay in tensor memory:
//   S^T = K Q^T, dP^T = V G^T, dV += P^T G, dK += dS^T Q
//   and the bias gradient: dS summed by bucket of the distance.
//
// delta.  g . out with the rounded out (and the weights rounded on its way)
// misses delta_i = sum_j p_ij dp_ij by about 2^-8 |g||out|, which is more than
// the other roundings where few keys carry a row (measured on histories of a
// few tokens: grad_q off by 0.0047 of its norm, 0.0017 being the result's own
// rounding).  With that estimate e, sum_j p (dp - e) = delta - e: dq sums its
// rows of dS in fp32, takes R times that sum off dQ (R needs little
// precision: the sum is small), and leaves the exact delta to dkv.  Where
// |lse| is large (kCoarse) it adds up the weights too, divides by their sum and
// leaves the sum's log2 to dkv (`excess`).
//
// A thread owns one row of S (a query in dq, a key in dkv) and half of a
// block's columns: a block takes two warpgroups.  head_dim <= 64: one set of
// score buffers, two CTAs per SM that fill each other's gaps (256 TMEM columns
// each).  Above: one CTA per SM (shared memory) with two sets of buffers and
// four warpgroups, two for the even and two for the odd blocks, so one block's
// products run beside the other's arithmetic.
//
// P and dS are rounded to the 16-bit type where they enter a product; the
// bias gradient sums the unrounded fp32 dS.  fp16's range is narrow (6e-8 to
// 65504), and dS moves with the upstream gradient: there dS is multiplied by the
// power of two that brings the largest |g| into [4, 8), of the row in dq and of
// the CTA's queries in dkv (a product's sum runs over them), and the results
// divided by it, both exactly.
#include <type_traits>

#include "attention_mma.cuh"

namespace tbe {

namespace {

template <int DP>
struct Shape {
    static constexpr int NB = DP == 64 ? 1 : 2;  // score buffers
    static constexpr int W = NB * 8;             // compute warps
    static constexpr int kThreads = W * 32 + 128;
    static constexpr int kPerSm = DP == 64 ? 2 : 1;
    static constexpr int kStages = 3;
    static constexpr int kBig = 128 * DP * 2;   // a 128-row tile
    static constexpr int kSmall = 64 * DP * 2;  // a 64-row tile
    static constexpr int a = 0, b = kBig, x = 2 * kBig, y = x + kStages * kSmall;
    static constexpr int table = y + kStages * kSmall;      // bias by distance: all, or 2 x 192 floats
    static constexpr int stat = table + kWholeEntries * 4;  // dkv: -lse, -delta and -excess, 2 x 3 x 64 floats
    static constexpr int sums = stat + 2 * 3 * 64 * 4;      // dkv: per warp, a sum per bucket
    static constexpr int diag = sums + W * kMaxBuckets * 4;       // dkv: per warp, 64 diagonals
    static constexpr int rows = sums;                             // dq: two row sums per thread
    static constexpr int dq_bytes = rows + 2 * W * 32 * 4 + 1024;
    static constexpr int dkv_bytes = diag + W * 64 * 4 + 1024;
    // TMEM columns: S (then P) and dP (then dS) per buffer, two accumulators
    static constexpr int cols = DP == 64 ? 256 : 512;
};

struct Bars {
    uint64_t big_full, fix[2], x_full[3], x_empty[3], y_full[3], y_empty[3], s_full[2], ds_full[2], t_full[2], t_empty[2],
        p_done, ds_done, last;
};

template <int NB>
__device__ __forceinline__ void init_bars(Bars& b) {
    mbar_init(&b.big_full, 2);
    for (int i = 0; i < 3; ++i) {
        mbar_init(&b.x_full[i], 1);
        mbar_init(&b.x_empty[i], 1);
        mbar_init(&b.y_full[i], 1);
        mbar_init(&b.y_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
        mbar_init(&b.s_full[i], 1);
        mbar_init(&b.ds_full[i], 8);
        mbar_init(&b.t_full[i], 1);
        mbar_init(&b.t_empty[i], 8);
        mbar_init(&b.fix[i], 1);
    }
    mbar_init(&b.p_done, 1);
    mbar_init(&b.ds_done, 1);
    mbar_init(&b.last, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
}

// A loader warp: its 128-row tile, then the 64-row tiles of the ring.
template <int DP, typename F>
__device__ __forceinline__ bool run_loader(unsigned char* big, const TileMap& big_map, int big_head, int big_first,
                                           unsigned char* ring, const TileMap& map, uint64_t* big_full,
                                           uint64_t* full, uint64_t* empty, uint64_t* fix, const AttnItem& it,
                                           int steps, int lane, F place) {
    uint32_t phase = 0;
    return load_tile<128, DP>(big, big_map, it, big_head, big_first, big_full, fix, phase, lane) &&
           load_ring<DP, Shape<DP>::kStages>(ring, map, it, full, empty, fix, phase, steps, lane, place);
}

// The product warp of both kernels.  Per block n: S = A X^T and dP = B Y^T
// into its buffer; once P and dS stand there, first += P Z and second += dS X,
// where Z is X (dq) or Y (dkv).  Block n + NB's scores overwrite P and dS, so
// each waits for its product; the next tiles' wait and the first product's
// are hidden behind the second product, the second's behind S.
template <int DT, int DP, bool ZisX>
__device__ __forceinline__ bool run_products(Bars& bars, uint32_t sbase, uint32_t tmem, uint32_t t_first,
                                             uint32_t t_second, int ksteps, int steps) {
    using L = Shape<DP>;
    constexpr int NB = L::NB;
    const uint32_t id_s = mma_idesc(DT == DT_BF16, 128, 64);
    const uint32_t id_o = mma_idesc(DT == DT_BF16, 128, ksteps * 16) | kMnMajorB;
    const uint64_t da = smem_desc_sw128(sbase + L::a, 1024), db = smem_desc_sw128(sbase + L::b, 1024);
    const uint64_t dx = smem_desc_sw128(sbase + L::x, 1024), dy = smem_desc_sw128(sbase + L::y, 1024);
    const uint64_t mx = smem_desc_mn(sbase + L::x, 64 * 128), my = smem_desc_mn(sbase + L::y, 64 * 128);
    auto wait = [&](uint64_t* bar, int phase) {
        const bool in = mbar_wait_tight(bar, phase & 1);
        const bool all = __all_sync(0xffffffffu, in);
        tcgen05_after_sync();
        return all;
    };
    auto tiles_in = [&](int n) {
        return wait(&bars.x_full[n % L::kStages], n / L::kStages) && wait(&bars.y_full[n % L::kStages], n / L::kStages);
    };
    auto issue_dp = [&](int n) {
        const int st = n % L::kStages;
        issue_scores<DP>(tmem + (n % NB) * 128 + 64, db, dy + st * (L::kSmall / 16), id_s, ksteps);
        if (ZisX && n + L::kStages < steps) mma_commit(&bars.y_empty[st]);
        mma_commit(&bars.s_full[n % NB]);
    };
    auto issue_s = [&](int n) {
        issue_scores<DP>(tmem + (n % NB) * 128, da, dx + n % L::kStages * (L::kSmall / 16), id_s, ksteps);
    };
    if (!wait(&bars.big_full, 0)) return false;
    for (int n = 0; n < NB && n < steps; ++n) {
        if (!tiles_in(n)) return false;
        if (elect_one()) {
            issue_s(n);
            issue_dp(n);
        }
        __syncwarp();
    }
    for (int n = 0; n < steps; ++n) {
        const int st = n % L::kStages;
        const uint32_t t = tmem + (n % NB) * 128;
        const bool more = n + NB < steps;
        if (!wait(&bars.ds_full[n % NB], n / NB)) return false;
        if (elect_one()) {
            issue_product<16>(t_first, t, (ZisX ? mx : my) + st * (L::kSmall / 16), id_o, n > 0);
            if (!ZisX && n + L::kStages < steps) mma_commit(&bars.y_empty[st]);
            if (more) mma_commit(&bars.p_done);
            issue_product<16>(t_second, t + 64, mx + st * (L::kSmall / 16), id_o, n > 0);
            if (n + L::kStages < steps) mma_commit(&bars.x_empty[st]);
            if (more) mma_commit(&bars.ds_done);
            if (n + 1 == steps) mma_commit(&bars.last);
        }
        __syncwarp();
        if (more) {
            if (!tiles_in(n + NB) || !wait(&bars.p_done, n)) return false;
            if (elect_one()) issue_s(n + NB);
            __syncwarp();
            if (!wait(&bars.ds_done, n)) return false;
            if (elect_one()) issue_dp(n + NB);
            __syncwarp();
        }
    }
    return true;
}

// The helper warp's table of one block: entry x is the bias (base 2) at
// distance least + x, 191 of them; nothing where all share one bucket.
// Returns whether they do, and that bucket's bias.
template <int DT>
__device__ __forceinline__ bool spread_bias(float* bt, const AttnShape& s, const void* bias, int head, int least,
                                            int lane, float& same, int& bucket) {
    bucket = attn_bucket(s, tmax(0, least));
    const int b1 = attn_bucket(s, tmax(0, least + 190));
    same = bias_base2(load_elem<DT>(bias, (int64_t)bucket * s.H + head));
    if (bucket == b1) return true;
    for (int x = lane; x < 191; x += 32) {
        const int d = least + x;
        bt[x] = d >= 0 ? bias_base2(load_elem<DT>(bias, (int64_t)attn_bucket(s, d) * s.H + head)) : 0.f;
    }
    return false;
}

// ------------------------------------------------------------------- dq

template <int DT, int DP>
__global__ void __launch_bounds__(Shape<DP>::kThreads, Shape<DP>::kPerSm) attn_dq_mma_kernel(const AttnBackward p,
                                                                                                   const __grid_constant__ AttnMaps maps) {
    using L = Shape<DP>;
    constexpr int NB = L::NB, kHelp = L::W;  // first helper warp: products; then loaders K, V; then bias
    constexpr bool kUnits = DT == DT_F16;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ Bars bars;
    __shared__ uint32_t tmem_slot;
    __shared__ float same_bias[2];
    __shared__ int several[2];  // the block's distances have several buckets

    const int64_t w = blockIdx.x / p.s.H;
    const int head = (int)(blockIdx.x % p.s.H);
    AttnItem it;
    if (!find_item(p.src, w, it)) return;
    const int kvh = head / p.s.G, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int first = it.tile * 128, D = p.s.D, ksteps = (D + 15) / 16;
    const int hi = tmin(first + 127, it.len - 1) / 64 + 1;
    const int64_t from = (int64_t)first - p.s.window + 1;
    const int lo = from > 0 ? (int)(from / 64) : 0;
    const int sink_blocks = tmin((p.s.sinks + 63) / 64, lo);
    const int steps = sink_blocks + hi - lo;
    auto block_of = [&](int n) { return n < sink_blocks ? n : lo + n - sink_blocks; };

    const uint32_t sbase = smem_u32(smem);
    if (threadIdx.x == 0) init_bars<NB>(bars);
    if (warp == kHelp) tmem_alloc(&tmem_slot, L::cols);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = tmem_slot;
    const uint32_t t_dq = tmem + NB * 128, t_r = t_dq + DP;  // S at buf*128, dP at buf*128 + 64
    bool ok = true;
    const bool whole = keep_whole(p.s);

    if (warp == kHelp) {
        // R += P K, dQ += dS K
        ok = run_products<DT, DP, true>(bars, sbase, tmem, t_r, t_dq, ksteps, steps);
    } else if (warp == kHelp + 1) {
        ok = run_loader<DP>(smem + L::a, maps.q, head, first, smem + L::x, maps.k, &bars.big_full, bars.x_full,
                            bars.x_empty, &bars.fix[0], it, steps, lane,
                            [&](int n) { return make_int2(block_of(n) * 64, kvh); });
    } else if (warp == kHelp + 2) {
        ok = run_loader<DP>(smem + L::b, maps.g, head, first, smem + L::y, maps.v, &bars.big_full, bars.y_full,
                            bars.y_empty, &bars.fix[1], it, steps, lane,
                            [&](int n) { return make_int2(block_of(n) * 64, kvh); });
    } else if (warp == kHelp + 3) {
        if (p.bias && !whole) {
            float* bt = reinterpret_cast<float*>(smem + L::table);
            for (int n = 0; n < steps; ++n) {
                const int buf = n & 1;
                if (n >= 2) ok = mbar_wait_tight(&bars.t_empty[buf], ((n / 2) - 1) & 1);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                float same;
                int bucket;
                const bool one = spread_bias<DT>(bt + buf * 192, p.s, p.bias, head, first - block_of(n) * 64 - 63, lane,
                                                 same, bucket);
                if (lane == 0) {
                    same_bias[buf] = same;
                    several[buf] = !one;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.t_full[buf]);
            }
        }
    } else {
        const int wg = warp / 4, half = wg % 2, q4 = warp % 4, row = q4 * 32 + lane, i = first + row;
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        const float c2 = p.s.scale * kLog2e;
        float* bt = reinterpret_cast<float*>(smem + L::table);
        const bool wait_bias = p.bias && !whole;
        const float last_bias = last_bias_of<DT>(p.s, p.bias, head);
        if (p.bias && whole) fill_bias<DT>(bt, p.s, p.bias, head, first + 127, threadIdx.x, L::W * 32);
        float less = -INFINITY, delta = 0.f, size = 0.f;  // size: the largest |g|
        if (i < it.len) {
            const int64_t at = (int64_t)head * p.N + it.start + i;
            const float x = p.lse[at];
            less = attn_no_weights(x) ? -INFINITY : -x;  // then all its weights are 2^-inf
            if constexpr (L::kPerSm == 1) {
                delta = p.delta[at];
                if constexpr (kUnits) size = p.size[at];
            } else {
                // the estimate of delta, g . out: half of the columns each warpgroup
                const int64_t token = (int64_t)it.start + i;
                const uint16_t* g =
                    static_cast<const uint16_t*>(p.g.data) + token * p.g.token_stride + head * p.g.head_stride;
                const uint16_t* o = static_cast<const uint16_t*>(p.out) + (token * p.s.H + head) * D;
#pragma unroll
                for (int c = 0; c < 32; c += 8) {
                    const int col = wg * 32 + c;
                    if (col >= D) break;
                    float u[8], v[8];
                    unpack16<DT>(__ldg(reinterpret_cast<const uint4*>(g + col)), u);
                    unpack16<DT>(__ldg(reinterpret_cast<const uint4*>(o + col)), v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        delta = fmaf(u[e], v[e], delta);
                        if constexpr (kUnits) size = fmaxf(size, fabsf(u[e]));
                    }
                }
            }
        }
        float* rows = reinterpret_cast<float*>(smem + L::rows);
        if constexpr (L::kPerSm > 1) {
            rows[wg * 128 + row] = delta;
            rows[(2 + wg) * 128 + row] = size;
            asm volatile("bar.sync 1, %0;" ::"n"(L::W * 32) : "memory");
            delta = rows[row] + rows[128 + row];
            size = fmaxf(rows[256 + row], rows[384 + row]);
            if constexpr (kUnits)
                if (wg == 0 && i < it.len) p.size[(int64_t)head * p.N + it.start + i] = size;
        }
        const float unit = kUnits ? attn_unit(size) : 1.f;
        asm volatile("bar.sync 1, %0;" ::"n"(L::W * 32) : "memory");  // the table stands; rows is free again
        float sum0 = 0.f, sum1 = 0.f;  // of the row's dS
        // the blocks' loop, for warps with a row whose weights have to be added
        // up and for the others (a test in the loop costs the latter 5 %)
        const bool large = fabsf(less) >= kCoarse && less > -INFINITY;
        float z0 = 0.f, z1 = 0.f;
        auto walk = [&](auto adds_up) {
            for (int n = wg / 2; n < steps; n += NB) {
                const int buf = n & 1, sb = n % NB;
                const uint32_t t_s = tmem + sb * 128 + lanes;
                ok = mbar_wait_tight(&bars.s_full[sb], (n / NB) & 1);
                if (ok && wait_bias) ok = mbar_wait_tight(&bars.t_full[buf], (n / 2) & 1);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tcgen05_after_sync();
                const int key0 = block_of(n) * 64;
                const bool table = p.bias && (whole ? first - key0 - 63 < p.s.far : several[buf] != 0);
                const float add = less + (wait_bias ? same_bias[buf] : last_bias);
                // whether the block holds a query whose only key is its own (attn_lone)
                const bool lone = (first == 0 && key0 == 0) || (p.s.window == 1 && p.s.sinks == 0);
                const bool all = key0 + 63 < first && (first + 127 - key0 < p.s.window || key0 + 63 < p.s.sinks);
                uint32_t pk[16], dk[16];
#pragma unroll
                for (int h = 0; h < 32; h += 16) {
                    float x[16], y[16];
                    tmem_ld16_pair(t_s + 32 * half + h, t_s + 64 + 32 * half + h, x, y);
                    const int key = key0 + 32 * half + h;
                    if (table) {
                        const float* b = bt + (whole ? i - key + 127 : buf * 192 + row + 63 - 32 * half - h);
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            float b0 = b[-c], b1 = b[-c - 1];
                            add2(b0, b1, less, less);
                            fma2(x[c], x[c + 1], c2, b0, b1);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; c += 2) fma2(x[c], x[c + 1], c2, add, add);
                    }
                    if (!all) {
                        const uint32_t seen =
                            bits_below(i - key + 1) &
                            (~bits_below(i - p.s.window + 1 - key) | bits_below(p.s.sinks - key));
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if (!(seen >> c & 1)) x[c] = -INFINITY;
                    }
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        x[c] = ex2(x[c]);
                        x[c + 1] = ex2(x[c + 1]);
                        if constexpr (kUnits)
                            fma2(y[c], y[c + 1], unit, -unit * delta, -unit * delta);
                        else
                            add2(y[c], y[c + 1], -delta, -delta);
                        mul2(y[c], y[c + 1], x[c], x[c + 1]);
                        pk[(h + c) / 2] = pack2<DT>(x[c], x[c + 1]);
                    }
                    if constexpr (decltype(adds_up)::value) {
#pragma unroll
                        for (int c = 0; c < 16; c += 2) add2(z0, z1, x[c], x[c + 1]);
                    }
                    if (lone) {
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if (key + c == i && attn_lone(i, i, p.s.window, p.s.sinks)) y[c] = 0.f;
                    }
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        dk[(h + c) / 2] = pack2<DT>(y[c], y[c + 1]);
                        add2(sum0, sum1, y[c], y[c + 1]);
                    }
                }
                // P and dS into the columns of S and dP that this thread has read
                tmem_st16(t_s + 32 * half, pk);
                tmem_st16(t_s + 64 + 32 * half, dk);
                tmem_wait_st();
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars.ds_full[sb]);
                    if (wait_bias) mbar_arrive(&bars.t_empty[buf]);
                }
            }
        };
        // (the usual one first: train full bf16 399 -> 394.5 us)
        if (!__any_sync(0xffffffffu, large))
            walk(std::false_type{});
        else
            walk(std::true_type{});
        if (ok) ok = mbar_wait_tight(&bars.last, 0);
        ok = __all_sync(0xffffffffu, ok);
        // delta - e of the row: all warpgroups' sums (every warp comes here)
        rows[wg * 128 + row] = sum0 + sum1;
        rows[(2 * NB + wg) * 128 + row] = z0 + z1;
        asm volatile("bar.sync 1, %0;" ::"n"(L::W * 32) : "memory");
        float over = 0.f, z = 0.f;
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k) {
            over += rows[k * 128 + row];
            z += rows[(2 * NB + k) * 128 + row];
        }
        const float inv = large ? 1.f / z : 1.f;
        over *= inv;
        if (ok) {
            tcgen05_after_sync();
            if (wg == 0 && i < it.len) {
                const int64_t at = (int64_t)head * p.N + it.start + i;
                p.delta[at] = delta + over * attn_unit_back(unit);
                if (large) p.excess[at] = log2f(z);
            }
            // dq = scale (dQ - over R) / z; the warpgroups take 32 columns each
            tmem_to_tile<DT>(smem + L::a, t_dq + lanes, wg * 32, row, p.s.scale * inv * attn_unit_back(unit),
                             t_r + lanes, -over);
        }
    }
    if (!ok) atomicOr(p.s.error, ERR_TIMEOUT);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp < 4) store_tile_rows<DP>(p.gq, smem + L::a, warp * 32, it.start, first, it.len, p.s.H, head, D, lane);
    if (warp == kHelp) tmem_dealloc(tmem, L::cols);
}

// ------------------------------------------------------------------ dkv

template <int DT, int DP>
__global__ void __launch_bounds__(Shape<DP>::kThreads, Shape<DP>::kPerSm) attn_dkv_mma_kernel(const AttnBackward p,
                                                                                                    const __grid_constant__ AttnMaps maps) {
    using L = Shape<DP>;
    constexpr int NB = L::NB, kHelp = L::W;
    constexpr bool kUnits = DT == DT_F16;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ Bars bars;
    __shared__ uint32_t tmem_slot;
    // -1: the block's distances have several; -2: and a query's excess is not in its -lse
    __shared__ int same_bucket[2];
    __shared__ uint32_t warp_size[L::kThreads / 32];  // fp16: the largest |g| that a warp saw

    // far items (the longest) first, then the tiles
    const int64_t turn = blockIdx.x / p.s.Hk;
    const int kvh = (int)(blockIdx.x % p.s.Hk);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int D = p.s.D, ksteps = (D + 15) / 16;
    AttnItem it;
    int64_t share;      // row of the bias gradient's shares
    int slot = -1;      // of the partial sums of the sinks' rows
    int first, qb0, blocks;
    const bool far = turn < p.far.most;
    if (far) {
        if (turn >= *p.far.n_items) return;
        const FarItem f = p.far.items[turn];
        it = AttnItem{f.start, f.len, 0, 0};
        share = p.max_items + turn;
        slot = f.slot + 1 + f.chunk;
        first = 0;
        qb0 = p.far.near + f.chunk * p.far.blocks;
        blocks = tmin(p.far.blocks, (it.len + 63) / 64 - qb0);
    } else {
        share = turn - p.far.most;
        if (!find_item(p.src, share, it)) return;
        const int kt = it.tiles - 1 - it.tile;  // the first tiles are seen most: they start first
        first = kt * 128;
        if (kt == 0 && p.far.most > 0) slot = p.far.slot_of[share];
        // query blocks that see a key of the tile
        const int64_t end = first < p.s.sinks ? it.len - 1 : tmin<int64_t>(it.len - 1, (int64_t)first + 126 + p.s.window);
        qb0 = first / 64;
        blocks = slot >= 0 ? p.far.near : (int)(end / 64) + 1 - qb0;
    }
    const int steps = blocks * p.s.G;  // for each head of the group
    auto place = [&](int n) { return make_int2((qb0 + n % blocks) * 64, kvh * p.s.G + n / blocks); };

    const uint32_t sbase = smem_u32(smem);
    if (threadIdx.x == 0) init_bars<NB>(bars);
    if (warp == kHelp) tmem_alloc(&tmem_slot, L::cols);
    float* sums = reinterpret_cast<float*>(smem + L::sums);
    for (int i = threadIdx.x; i < L::W * p.s.buckets; i += L::kThreads)
        sums[i / p.s.buckets * kMaxBuckets + i % p.s.buckets] = 0.f;
    if constexpr (kUnits) {  // the largest |g| of the CTA's queries and heads
        float size = 0.f;
        const int from = qb0 * 64, rows = tmin(it.len - from, blocks * 64);
        for (int g = 0; g < p.s.G; ++g) {
            const float* of = p.size + (int64_t)(kvh * p.s.G + g) * p.N + it.start + from;
#pragma unroll 4
            for (int r = threadIdx.x; r < rows; r += L::kThreads) size = fmaxf(size, of[r]);
        }
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(size));
        if (lane == 0) warp_size[warp] = most;
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    float unit = 1.f;
    if constexpr (kUnits) {
        uint32_t most = 0;
#pragma unroll
        for (int k = 0; k < L::kThreads / 32; ++k) most = tmax(most, warp_size[k]);
        unit = attn_unit(__uint_as_float(most));
    }
    const uint32_t tmem = tmem_slot;
    const uint32_t t_dk = tmem + NB * 128, t_dv = t_dk + DP;  // S^T at buf*128, dP^T at buf*128 + 64
    bool ok = true;

    if (warp == kHelp) {
        // dV += P^T G, dK += dS^T Q
        ok = run_products<DT, DP, false>(bars, sbase, tmem, t_dv, t_dk, ksteps, steps);
    } else if (warp == kHelp + 1) {
        ok = run_loader<DP>(smem + L::a, maps.k, kvh, first, smem + L::x, maps.q, &bars.big_full, bars.x_full,
                            bars.x_empty, &bars.fix[0], it, steps, lane, place);
    } else if (warp == kHelp + 2) {
        ok = run_loader<DP>(smem + L::b, maps.v, kvh, first, smem + L::y, maps.g, &bars.big_full, bars.y_full,
                            bars.y_empty, &bars.fix[1], it, steps, lane, place);
    } else if (warp == kHelp + 3) {
        // per query of the block: -lse (plus the bias less the excess where the
        // block has one bucket), delta and excess; the bias table else
        float* bt = reinterpret_cast<float*>(smem + L::table);
        float* stat = reinterpret_cast<float*>(smem + L::stat);
        for (int n = 0; n < steps; ++n) {
            const int buf = n & 1;
            if (n >= 2) ok = mbar_wait_tight(&bars.t_empty[buf], ((n / 2) - 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            const int2 at = place(n);
            float same = 0.f;
            bool one = true;
            int bucket = 0;
            if (p.bias) {
                const int least = at.x - first - 127;
                if (keep_whole(p.s)) {
                    same = last_bias_of<DT>(p.s, p.bias, at.y);
                    one = least >= p.s.far;
                    bucket = p.s.buckets - 1;
                } else {
                    one = spread_bias<DT>(bt + buf * 192, p.s, p.bias, at.y, least, lane, same, bucket);
                }
            }
            float x[2], delta[2], excess[2] = {0.f, 0.f};
            const int64_t k = (int64_t)at.y * p.N + it.start + at.x + lane;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const bool there = at.x + lane + 32 * c < it.len;
                x[c] = there ? p.lse[k + 32 * c] : -INFINITY;
                delta[c] = there ? p.delta[k + 32 * c] : 0.f;
            }
            const bool apart = __any_sync(0xffffffffu, attn_coarse(x[0]) || attn_coarse(x[1]));
            if (apart) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (attn_coarse(x[c])) excess[c] = p.excess[k + 32 * c];
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float less = attn_no_weights(x[c]) ? -INFINITY : one ? (same - x[c]) - excess[c] : -x[c];
                stat[buf * 192 + lane + 32 * c] = less;
                stat[buf * 192 + 64 + lane + 32 * c] = -unit * delta[c];
                if (apart) stat[buf * 192 + 128 + lane + 32 * c] = -excess[c];
            }
            if (lane == 0) same_bucket[buf] = one ? bucket : apart ? -2 : -1;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.t_full[buf]);
        }
    } else {
        const int wg = warp / 4, half = wg % 2, q4 = warp % 4, row = q4 * 32 + lane, j = first + row;
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        const float c2 = p.s.scale * kLog2e;
        float* mine = sums + warp * kMaxBuckets;
        float* diag = reinterpret_cast<float*>(smem + L::diag) + warp * 64;
        for (int g = 0; g < p.s.G; ++g) {
            float* bt = reinterpret_cast<float*>(smem + L::table);
            const bool whole = keep_whole(p.s);
            if (p.bias && whole) {
                fill_bias<DT>(bt, p.s, p.bias, kvh * p.s.G + g, (qb0 + blocks) * 64 - 1 - first, threadIdx.x, L::W * 32);
                asm volatile("bar.sync 1, %0;" ::"n"(L::W * 32) : "memory");
            }
            // the head's blocks, or every other one
            for (int n = g * blocks + (NB == 2 ? (g * blocks + wg / 2) % 2 : 0); n < (g + 1) * blocks && ok; n += NB) {
                const int buf = n & 1, sb = n % NB;
                const uint32_t t_s = tmem + sb * 128 + lanes;
                ok = mbar_wait_tight(&bars.s_full[sb], (n / NB) & 1);
                if (ok) ok = mbar_wait_tight(&bars.t_full[buf], (n / 2) & 1);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tcgen05_after_sync();
                const int q0 = place(n).x;
                const float* less = reinterpret_cast<const float*>(smem + L::stat) + buf * 192 + 32 * half;
                const int bucket = same_bucket[buf];
                const bool table = bucket < 0;
                float sum0 = 0.f, sum1 = 0.f, run = 0.f;
                // the warp's 32 x 32 pairs have 63 distances from `least` on: of
                // one bucket, of two (cut at column `cut` of the lane's row), or
                // of more.  Telling them apart pays where one CTA has the SM
                // (long window f16 backward 974 -> 932 us, its wide buckets
                // mostly one or two a warp); with two CTAs the longer code
                // costs more (train full bf16 320 -> 338), so there a block of
                // several buckets takes the general way.
                constexpr bool kTell = L::kPerSm == 1;
                const int least = q0 + 32 * half - first - 32 * q4 - 31;
                int low = bucket, high = table ? bucket + 2 : bucket, cut = 0;
                if (kTell && table) {
                    low = attn_bucket(p.s, tmax(0, least));
                    high = attn_bucket(p.s, tmax(0, least + 62));
                    if (high > low) cut = __ldg(p.s.starts + high) - (least + 31 - lane);
                }
                const bool all = q0 > first + 127 && (q0 + 63 - first < p.s.window || first + 127 < p.s.sinks);
                // whether the block holds a query whose only key is its own (attn_lone)
                const bool lone = !all && (q0 == 0 || (p.s.window == 1 && p.s.sinks == 0));
                uint32_t pk[16], dk[16];
#pragma unroll
                for (int h = 0; h < 32; h += 16) {
                    float x[16], y[16];
                    tmem_ld16_pair(t_s + 32 * half + h, t_s + 64 + 32 * half + h, x, y);
                    const int query = q0 + 32 * half + h;
                    const float* b = bt + (whole ? query - j + 127 : buf * 192 + 127 - row + 32 * half + h);
                    if (bucket == -2) {
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            const float b0 = (b[c] + less[h + c]) + less[128 + h + c];
                            const float b1 = (b[c + 1] + less[h + c + 1]) + less[128 + h + c + 1];
                            fma2(x[c], x[c + 1], c2, b0, b1);
                        }
                    } else if (table) {
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            const float4 t = *reinterpret_cast<const float4*>(less + h + c);
                            float b0 = b[c], b1 = b[c + 1], b2 = b[c + 2], b3 = b[c + 3];
                            add2(b0, b1, t.x, t.y);
                            add2(b2, b3, t.z, t.w);
                            fma2(x[c], x[c + 1], c2, b0, b1);
                            fma2(x[c + 2], x[c + 3], c2, b2, b3);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            const float4 t = *reinterpret_cast<const float4*>(less + h + c);
                            fma2(x[c], x[c + 1], c2, t.x, t.y);
                            fma2(x[c + 2], x[c + 3], c2, t.z, t.w);
                        }
                    }
                    if (!all) {
                        // query i sees key j: j <= i, and i < j + window or j a sink
                        const uint32_t seen =
                            ~bits_below(j - query) & bits_below(j < p.s.sinks ? INT_MAX : j + p.s.window - query);
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if (!(seen >> c & 1)) x[c] = -INFINITY;
                    }
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        const float4 t = *reinterpret_cast<const float4*>(less + 64 + h + c);
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[c + e] = ex2(x[c + e]);
                        if constexpr (kUnits) {
                            fma2(y[c], y[c + 1], unit, t.x, t.y);
                            fma2(y[c + 2], y[c + 3], unit, t.z, t.w);
                        } else {
                            add2(y[c], y[c + 1], t.x, t.y);
                            add2(y[c + 2], y[c + 3], t.z, t.w);
                        }
                        mul2(y[c], y[c + 1], x[c], x[c + 1]);
                        mul2(y[c + 2], y[c + 3], x[c + 2], x[c + 3]);
                        pk[(h + c) / 2] = pack2<DT>(x[c], x[c + 1]);
                        pk[(h + c) / 2 + 1] = pack2<DT>(x[c + 2], x[c + 3]);
                    }
                    if (lone) {
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if (query + c == j && attn_lone(j, j, p.s.window, p.s.sinks)) y[c] = 0.f;
                    }
#pragma unroll
                    for (int c = 0; c < 16; c += 2) dk[(h + c) / 2] = pack2<DT>(y[c], y[c + 1]);
                    if (p.bias && high == low) {
#pragma unroll
                        for (int c = 0; c < 16; c += 2) add2(sum0, sum1, y[c], y[c + 1]);
                    } else if (kTell && p.bias && high - low == 1) {
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if (h + c >= cut)
                                run += y[c];
                            else
                                sum0 += y[c];
                    } else if (p.bias) {
                        // column c has distance least + 31 - lane + c: a
                        // diagonal's sum moves one lane up a column and is
                        // complete at lane 31
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float t = __shfl_up_sync(0xffffffffu, run, 1);
                            run = y[c] + (lane == 0 ? 0.f : t);
                            if (lane == 31) diag[h + c] = run;
                        }
                    }
                }
                // P^T and dS^T into the columns of S^T and dP^T that this thread
                // has read
                tmem_st16(t_s + 32 * half, pk);
                tmem_st16(t_s + 64 + 32 * half, dk);
                tmem_wait_st();
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars.ds_full[sb]);
                    mbar_arrive(&bars.t_empty[buf]);
                }
                if (p.bias && (high == low || (kTell && high - low == 1))) {
                    float t = sum0 + sum1;  // the lower bucket's
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        t += __shfl_xor_sync(0xffffffffu, t, o);
                        if (kTell && high > low) run += __shfl_xor_sync(0xffffffffu, run, o);
                    }
                    if (lane == 0) {
                        mine[low] += t;
                        if (kTell && high > low) mine[high] += run;
                    }
                    __syncwarp();
                } else if (p.bias) {
                    // diag[x], x in [0, 63): distance least + x; the last
                    // column's running sums are the highest 32
                    if (lane < 31) diag[62 - lane] = run;
                    __syncwarp();
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        // sums of equal buckets, which are neighbours: a segmented
                        // scan over 32 distances, added by each segment's last lane
                        const int at = r * 32 + lane, d = least + at;
                        const int b = at < 63 && d >= 0 ? attn_bucket(p.s, d) : -1;
                        float t = b >= 0 ? diag[at] : 0.f;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const float tu = __shfl_up_sync(0xffffffffu, t, o);
                            const int bu = __shfl_up_sync(0xffffffffu, b, o);
                            if (lane >= o && bu == b) t += tu;
                        }
                        const int next = __shfl_down_sync(0xffffffffu, b, 1);
                        if (b >= 0 && (lane == 31 || next != b)) mine[b] += t;
                        __syncwarp();
                    }
                }
            }
            if (p.bias) {  // the head's share: all warps come here, whatever their waits said
                asm volatile("bar.sync 1, %0;" ::"n"(L::W * 32) : "memory");
                for (int b = threadIdx.x; b < p.s.buckets; b += L::W * 32) {
                    float t = 0.f;
                    for (int k = 0; k < L::W; ++k) {
                        t += sums[k * kMaxBuckets + b];
                        sums[k * kMaxBuckets + b] = 0.f;
                    }
                    p.bias_part[(share * p.s.H + kvh * p.s.G + g) * p.s.buckets + b] = t * attn_unit_back(unit);
                }
                asm volatile("bar.sync 1, %0;" ::"n"(L::W * 32) : "memory");
            }
        }
        if (ok) ok = mbar_wait_tight(&bars.last, 0);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
            tcgen05_after_sync();
            // dk into K's tile, dv into V's: 64 columns a warpgroup
            const bool of_v = wg / NB == 1;
            const float back = of_v ? 1.f : attn_unit_back(unit);
            if (slot >= 0 && q4 * 32 < p.s.sinks) {
                float* to = p.far.part + ((((int64_t)slot * p.s.Hk + kvh) * 2 + of_v) * p.s.sinks + row) * DP + (wg % NB) * 64;
#pragma unroll
                for (int c = 0; c < 64; c += 16) {
                    float o[16];
                    tmem_ld16((of_v ? t_dv : t_dk) + lanes + (wg % NB) * 64 + c, o);
                    if (row < p.s.sinks)
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<float4*>(to + c + e) =
                                make_float4(o[e] * back, o[e + 1] * back, o[e + 2] * back, o[e + 3] * back);
                }
            }
#pragma unroll
            for (int c = 0; c < 64; c += 32)
                tmem_to_tile<DT>(smem + (of_v ? L::b : L::a), (of_v ? t_dv : t_dk) + lanes, (wg % NB) * 64 + c, row,
                                 of_v ? 1.f : p.s.scale * back);
        }
    }
    if (!ok) atomicOr(p.s.error, ERR_TIMEOUT);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (far) {
        // the join writes the sinks' rows
    } else if (warp < 4)
        store_tile_rows<DP>(p.gk, smem + L::a, warp * 32, it.start, first, it.len, p.s.Hk, kvh, D, lane);
    else if (warp < 8)
        store_tile_rows<DP>(p.gv, smem + L::b, (warp - 4) * 32, it.start, first, it.len, p.s.Hk, kvh, D, lane);
    if (warp == kHelp) tmem_dealloc(tmem, L::cols);
}

// The sinks' rows of a split history: the tile's own sums and its far chunks',
// in their order, rounded once.
template <int DT, int DP>
__global__ void __launch_bounds__(256) attn_far_join_kernel(const AttnBackward p) {
    const int turn = blockIdx.x / p.s.Hk, kvh = blockIdx.x % p.s.Hk;
    if (turn >= *p.far.n_items) return;
    const FarItem f = p.far.items[turn];
    if (f.chunk != 0) return;
    const int64_t stride = (int64_t)p.s.Hk * 2 * p.s.sinks * DP;
    for (int i = threadIdx.x; i < 2 * p.s.sinks * DP; i += 256) {
        const int col = i % DP, row = i / DP % p.s.sinks, of_v = i / DP / p.s.sinks;
        if (col >= p.s.D) continue;
        const float* from = p.far.part + f.slot * stride + (int64_t)kvh * 2 * p.s.sinks * DP + i;
        float t = 0.f;
        for (int c = 0; c <= f.chunks; ++c) t += from[c * stride];
        const int64_t at = (((int64_t)f.start + row) * p.s.Hk + kvh) * p.s.D + col;
        if (of_v)
            store_elem<DT>(p.gv, at, t);
        else
            store_elem<DT>(p.gk, at, t * p.s.scale);
    }
}

// delta_i = g_i . out_i of every (token, head), and in fp16 the largest |g|: eight lanes a row, 16 bytes a
// lane and step.  Memory-bound (each row of g and out is read once).  For
// head_dim > 64 only: there dq runs one CTA per SM and shows every microsecond
// of its start (long window f16 backward 1082 us with this kernel, 1133 with
// dq's own loads); with two, dq's own loads save the launch and the pass
// (train full bf16 337 -> 324).
template <int DT>
__global__ void __launch_bounds__(256) attn_delta_kernel(const AttnBackward p) {
    const int64_t r = (int64_t)blockIdx.x * 32 + threadIdx.x / 8;
    const int chunk = threadIdx.x % 8;
    const int64_t token = r / p.s.H;
    const int head = (int)(r % p.s.H);
    float t = 0.f, size = 0.f;
    if (token < p.N) {
        const uint16_t* g = static_cast<const uint16_t*>(p.g.data) + token * p.g.token_stride + head * p.g.head_stride;
        const uint16_t* o = static_cast<const uint16_t*>(p.out) + r * p.s.D;
        for (int c = chunk * 8; c < p.s.D; c += 64) {
            float x[8], y[8];
            unpack16<DT>(__ldg(reinterpret_cast<const uint4*>(g + c)), x);
            unpack16<DT>(__ldg(reinterpret_cast<const uint4*>(o + c)), y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t = fmaf(x[e], y[e], t);
                size = fmaxf(size, fabsf(x[e]));
            }
        }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
        t += __shfl_xor_sync(0xffffffffu, t, o);
        if constexpr (DT == DT_F16) size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, o));
    }
    if (chunk == 0 && token < p.N) {
        p.delta[(int64_t)head * p.N + token] = t;
        if constexpr (DT == DT_F16) p.size[(int64_t)head * p.N + token] = size;
    }
}

template <int DT, int DP>
cudaError_t launch(const AttnBackward& p, const AttnMaps& maps, int64_t max_items, cudaStream_t s) {
    using L = Shape<DP>;
    cudaError_t e = cudaSuccess;
    if constexpr (L::kPerSm == 1) {
        attn_delta_kernel<DT><<<(unsigned)((p.N * p.s.H + 31) / 32), 256, 0, s>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    attn_dq_mma_kernel<DT, DP><<<(unsigned)(max_items * p.s.H), L::kThreads, L::dq_bytes, s>>>(p, maps);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    attn_dkv_mma_kernel<DT, DP>
        <<<(unsigned)((p.far.most + max_items) * p.s.Hk), L::kThreads, L::dkv_bytes, s>>>(p, maps);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.far.most == 0) return e;
    attn_far_join_kernel<DT, DP><<<(unsigned)(p.far.most * p.s.Hk), 256, 0, s>>>(p);
    return cudaGetLastError();
}

template <int DT, int DP>
cudaError_t configure() {
    const cudaError_t e = cudaFuncSetAttribute(attn_dq_mma_kernel<DT, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Shape<DP>::dq_bytes);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(attn_dkv_mma_kernel<DT, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Shape<DP>::dkv_bytes);
}

}  // namespace

cudaError_t attn_backward_mma_configure() {
    cudaError_t e = configure<DT_F16, 64>();
    if (e == cudaSuccess) e = configure<DT_F16, 128>();
    if (e == cudaSuccess) e = configure<DT_BF16, 64>();
    if (e == cudaSuccess) e = configure<DT_BF16, 128>();
    return e;
}

cudaError_t launch_attn_backward_mma(const AttnBackward& p, const AttnMaps& maps, int64_t max_items, cudaStream_t s) {
    if (p.s.dtype == DT_F16) return p.s.D <= 64 ? launch<DT_F16, 64>(p, maps, max_items, s) : launch<DT_F16, 128>(p, maps, max_items, s);
    return p.s.D <= 64 ? launch<DT_BF16, 64>(p, maps, max_items, s) : launch<DT_BF16, 128>(p, maps, max_items, s);
}

}  // namespace tbe
