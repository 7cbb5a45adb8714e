// Attention over ragged histories on the tensor cores (tcgen05), forward.
//
// One CTA takes 128 queries of one history and head and walks the visible
// keys in blocks of 64:
//   S = Q K^T           (128 x 64, both operands in shared memory, fp32 in TMEM)
//   P = 2^(S c + b - m) (one query per thread, rounded to the 16-bit type, TMEM)
//   O += P V            (P from TMEM, V as stored: its MN-major descriptor)
// Roles: warps 0-3 softmax (thread = query), warp 4 issues the products,
// warps 5 and 6 fetch the tiles (TMA), warp 7 spreads the bias over the
// block's distances where the table of all distances is too large to keep.  S has two
// buffers, so the next block's scores are computed while this one's softmax
// runs; P takes its S's place.  Two CTAs share an SM (256 TMEM columns each)
// and fill each other's gaps.
//
// The running maximum m is only moved when a score exceeds it by 2^8
// (kLazy): the weights then stay below 256, exact in fp32 sums and within
// fp16's range, and the accumulator is rescaled rarely.
//
// A batch of many histories whose tokens see few keys has many tiles of few
// blocks: there two CTAs per SM take the (tile, head) items in turn, so that the
// next one's tiles are fetched and its first scores computed under the last
// one's softmax (12 % on 512 ragged bf16 histories, 78 us now).  Else each item
// gets a CTA, which the hardware hands out as others end (the call's rule has
// both sides' times).
//
// The weights are rounded to the 16-bit type for the second product (the
// tensor cores' operand type); their sum is kept unrounded in fp32.
#include <type_traits>

#include "attention_mma.cuh"

namespace tbe {

namespace {

constexpr int kThreads = 256;
constexpr float kLazy = 8.f;

template <int DP>
struct Fwd {
    static constexpr int kStages = DP == 64 ? 3 : 2;
    static constexpr int kQs = DP == 64 ? 2 : 1;   // query tiles
    static constexpr int kTile = 64 * DP * 2;  // bytes of a K or V tile
    static constexpr int kQ = 128 * DP * 2;
    static constexpr int q = 0, k = kQs * kQ, v = k + kStages * kTile, bias = v + kStages * kTile;
    static constexpr int bytes = bias + kWholeEntries * 4 + 1024;  // 1024: the swizzle's alignment
    static constexpr int cols = 256;
};

struct FwdBars {
    uint64_t q_full[2], q_empty[2], fix[2], k_full[3], k_empty[3], v_full[3], v_empty[3], s_full[2], p_full[2], o_done,
        o_last, o_free, b_full[2], b_empty[2];
};

// Whether any thread of the four softmax warps says so; they all wait for it.
__device__ __forceinline__ bool softmax_warps_any(bool x) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)x)
        : "memory");
    return any != 0;
}

// One (query tile, head) and the key blocks it sees: [0, sinks) and
// [lo, lo + steps - sinks).
struct Turn {
    AttnItem it;
    int head, kvh, first, lo, sinks, steps;
    __device__ __forceinline__ int block(int n) const { return n < sinks ? n : lo + n - sinks; }
};

__device__ __forceinline__ bool take(const AttnForward& p, int64_t w, Turn& t) {
    if (!find_item(p.src, w / p.s.H, t.it)) return false;
    t.head = (int)(w % p.s.H);
    t.kvh = t.head / p.s.G;
    t.first = t.it.tile * 128;
    const int hi = tmin(t.first + 127, t.it.len - 1) / 64 + 1;
    const int64_t from = (int64_t)t.first - p.s.window + 1;
    t.lo = from > 0 ? (int)(from / 64) : 0;
    t.sinks = tmin((p.s.sinks + 63) / 64, t.lo);
    t.steps = t.sinks + hi - t.lo;
    return true;
}

// TURNS: the grid is two CTAs per SM, which take the items in turn.
template <int DT, int DP, bool TURNS>
__global__ void __launch_bounds__(kThreads, 2)
    attn_fwd_mma_kernel(const AttnForward p, const __grid_constant__ AttnMaps maps) {
    using L = Fwd<DP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ FwdBars bars;
    __shared__ uint32_t tmem_slot;
    __shared__ float uniform_bias[2];
    __shared__ int is_uniform[2];

    int64_t w = blockIdx.x;
    Turn t;
    if (!take(p, w, t)) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int D = p.s.D, ksteps = (D + 15) / 16;
    // every role walks the CTA's turns by itself, with its own counts of blocks
    // and turns: a loader is ahead of the products, the products of the softmax
    auto more = [&]() {
        if constexpr (!TURNS) return false;
        w += gridDim.x;
        return take(p, w, t);
    };

    const uint32_t sbase = smem_u32(smem);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bars.k_full[i], 1);
            mbar_init(&bars.k_empty[i], 1);
            mbar_init(&bars.v_full[i], 1);
            mbar_init(&bars.v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.q_full[i], 1);
            mbar_init(&bars.q_empty[i], 4);
            mbar_init(&bars.fix[i], 1);
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i], 4);
            mbar_init(&bars.b_full[i], 1);
            mbar_init(&bars.b_empty[i], 4);
        }
        mbar_init(&bars.o_done, 1);
        mbar_init(&bars.o_last, 1);
        mbar_init(&bars.o_free, 4);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (warp == 4) tmem_alloc(&tmem_slot, L::cols);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = tmem_slot;
    const uint32_t t_o = tmem + 128;  // S0 and S1 at columns 0 and 64
    bool ok = true;
    if (warp == 5 || warp == 6) {
        // ---- loaders: warp 5 Q and K, warp 6 V
        uint32_t fix_phase = 0;
        int done = 0, turn = 0;
        do {
            auto place = [&](int n) { return make_int2(t.block(n) * 64, t.kvh); };
            if (warp == 5) {
                const int qb = turn % L::kQs;
                ok = turn < L::kQs || mbar_wait_tight(&bars.q_empty[qb], (turn / L::kQs - 1) & 1);
                ok = __all_sync(0xffffffffu, ok) &&
                     load_tile<128, DP>(smem + L::q + qb * L::kQ, maps.q, t.it, t.head, t.first, &bars.q_full[qb],
                                        &bars.fix[0], fix_phase, lane) &&
                     load_ring<DP, L::kStages>(smem + L::k, maps.k, t.it, bars.k_full, bars.k_empty, &bars.fix[0],
                                               fix_phase, t.steps, lane, place, done);
            } else {
                ok = load_ring<DP, L::kStages>(smem + L::v, maps.v, t.it, bars.v_full, bars.v_empty, &bars.fix[1],
                                               fix_phase, t.steps, lane, place, done);
            }
            done += t.steps;
            ++turn;
        } while (ok && more());
    } else if (warp == 7) {
        // ---- bias by distance, where the table of all distances is not kept:
        // entry x of the block's table is the bias at distance base + x - 63,
        // x in [0, 191)
        if (p.bias && !keep_whole(p.s)) {
            float* bt = reinterpret_cast<float*>(smem + L::bias);
            int done = 0;
            do {
                for (int n = 0; n < t.steps && ok; ++n, ++done) {
                    const int buf = done & 1;
                    if (done >= 2) ok = mbar_wait_tight(&bars.b_empty[buf], (done / 2 - 1) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const int base = t.first - t.block(n) * 64;
                    const int least = tmax(0, base - 63), most = base + 127;
                    const int b0 = attn_bucket(p.s, least), b1 = attn_bucket(p.s, tmax(most, 0));
                    if (lane == 0) {
                        is_uniform[buf] = b0 == b1;
                        uniform_bias[buf] = bias_base2(load_elem<DT>(p.bias, (int64_t)b0 * p.s.H + t.head));
                    }
                    if (b0 != b1)
                        for (int x = lane; x < 191; x += 32) {
                            const int d = base + x - 63;
                            bt[buf * 192 + x] =
                                d >= 0 ? bias_base2(load_elem<DT>(p.bias, (int64_t)attn_bucket(p.s, d) * p.s.H + t.head))
                                       : 0.f;
                        }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.b_full[buf]);
                }
            } while (ok && more());
        }
    } else if (warp == 4) {
        // ---- products
        const uint32_t id_s = mma_idesc(DT == DT_BF16, 128, 64);
        const uint32_t id_o = mma_idesc(DT == DT_BF16, 128, ksteps * 16) | kMnMajorB;
        const uint64_t dq = smem_desc_sw128(sbase + L::q, 1024), dk = smem_desc_sw128(sbase + L::k, 1024);
        const uint64_t dv = smem_desc_mn(sbase + L::v, 64 * 128);
        auto wait = [&](uint64_t* bar, int phase) {
            const bool in = mbar_wait_tight(bar, phase & 1);
            const bool all = __all_sync(0xffffffffu, in);
            tcgen05_after_sync();
            return all;
        };
        int g = 0, turn = 0, last = 0;  // blocks before this turn, turns, o_done's phases before this turn
        do {
            const int steps = t.steps, qb = turn % L::kQs;
            auto scores = [&](int n) {
                const int st = (g + n) % L::kStages;
                if (!wait(&bars.k_full[st], (g + n) / L::kStages)) return false;
                if (elect_one()) {
                    issue_scores<DP>(tmem + ((g + n) & 1) * 64, dq + qb * (L::kQ / 16), dk + st * (L::kTile / 16), id_s,
                                     ksteps);
                    mma_commit(&bars.k_empty[st]);
                    mma_commit(&bars.s_full[(g + n) & 1]);
                }
                __syncwarp();
                return true;
            };
            // the first block's scores take the place of the last turn's last
            // but one weights, the second's of its last; and this turn's O the
            // last's, once the softmax has read it
            ok = wait(&bars.q_full[qb], turn / L::kQs) && scores(0) && (turn == 0 || wait(&bars.o_last, turn - 1)) &&
                 (steps == 1 || scores(1)) && (turn == 0 || wait(&bars.o_free, turn - 1));
            for (int n = 0; n < steps && ok; ++n) {
                const int st = (g + n) % L::kStages;
                ok = wait(&bars.v_full[st], (g + n) / L::kStages) && wait(&bars.p_full[(g + n) & 1], (g + n) / 2);
                if (!ok) break;
                if (elect_one()) {
                    issue_product(t_o, tmem + ((g + n) & 1) * 64, dv + st * (L::kTile / 16), id_o, n > 0);
                    mma_commit(&bars.v_empty[st]);
                    mma_commit(n + 1 < steps ? &bars.o_done : &bars.o_last);
                }
                __syncwarp();
                // block n + 2's scores overwrite P(n): wait for its product
                if (n + 2 <= steps) ok = wait(&bars.o_done, last + n) && (n + 2 == steps || scores(n + 2));
            }
            g += steps;
            last += steps - 1;
            ++turn;
        } while (ok && more());
        // nothing of this CTA arrives on a barrier after its end
        if (ok)
            ok = wait(&bars.k_empty[(g - 1) % L::kStages], (g - 1) / L::kStages) &&
                 wait(&bars.v_empty[(g - 1) % L::kStages], (g - 1) / L::kStages);
    } else {
        // ---- softmax: thread = query
        const int row = threadIdx.x;
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const float c2 = p.s.scale * kLog2e;
        float* bt = reinterpret_cast<float*>(smem + L::bias);
        int g = 0, turn = 0, last = 0, held = -1;  // held: the head whose bias the kept table has
        float last_bias = 0.f;
        const bool whole = keep_whole(p.s), wait_bias = p.bias && !whole;
        bool coarse = false;  // the head has a bias of large magnitude
        do {
            const int steps = t.steps, first = t.first, i = first + row;
            if (p.bias && t.head != held) {
                last_bias = last_bias_of<DT>(p.s, p.bias, t.head);
                bool large = false;
                if (whole) {
                    asm volatile("bar.sync 1, 128;" ::: "memory");  // the last table is read
                    large = fill_bias<DT>(bt, p.s, p.bias, t.head, TURNS ? INT_MAX / 2 : first + 127, row, 128);
                } else {
                    for (int b = row; b < p.s.buckets; b += 128)
                        large |= attn_coarse(bias_base2(load_elem<DT>(p.bias, (int64_t)b * p.s.H + t.head)));
                }
                coarse = softmax_warps_any(large);  // (and the table stands)
                held = t.head;
            }
            float off = 0.f;  // taken off the row's biases
            if (coarse)
                off = attn_bias_off(attn_bias_top(p.s, i, 0, 1, [&](int b) {
                    return bias_base2(load_elem<DT>(p.bias, (int64_t)b * p.s.H + t.head));
                }));
            float m = -INFINITY, l0 = 0.f, l1 = 0.f;
            // the blocks' loop, with biases less `off` and without (a register
            // and a test more in the latter cost 4 %)
            auto walk = [&](auto shifts) {
                constexpr bool kShifts = decltype(shifts)::value;
                for (int n = 0; n < steps && ok; ++n) {
                    const int buf = (g + n) & 1;
                    const uint32_t t_s = tmem + buf * 64 + lanes;
                    ok = mbar_wait_tight(&bars.s_full[buf], ((g + n) / 2) & 1);
                    if (ok && wait_bias) ok = mbar_wait_tight(&bars.b_full[buf], ((g + n) / 2) & 1);
                    // products up to n - 2 have completed (their P's place is S(n)'s,
                    // which is full); n - 1 is waited for where O is touched
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    tcgen05_after_sync();
                    float x[64];
                    tmem_ld32_issue(t_s, x);
                    tmem_ld32_issue(t_s + 32, x + 32);
                    tmem_wait_ld(x, 64);
                    const int key0 = t.block(n) * 64;
                    const bool table = p.bias && (whole ? first - key0 - 63 < p.s.far : !is_uniform[buf]);
                    // logit = x * by + add: with a table it is formed here, else (one
                    // bias for the block, and c2 > 0) the maximum is taken of the raw
                    // products and one multiply-add before ex2 does it all
                    float by = c2, add = wait_bias ? uniform_bias[buf] : last_bias;
                    if (table) {
                        const float* b = bt + (whole ? i - key0 + 127 : buf * 192 + row + 63);
                        if constexpr (kShifts) {
#pragma unroll
                            for (int c = 0; c < 64; c += 2) fma2(x[c], x[c + 1], c2, b[-c] - off, b[-c - 1] - off);
                        } else {
#pragma unroll
                            for (int c = 0; c < 64; c += 2) fma2(x[c], x[c + 1], c2, b[-c], b[-c - 1]);
                        }
                        by = 1.f;
                        add = 0.f;
                    } else if (add == -FLT_MAX) {
                        // a bias that swallows the logits (a type's lowest value):
                        // one rounding of the two, as in a table's addition
#pragma unroll
                        for (int c = 0; c < 64; c += 2)
                            fma2(x[c], x[c + 1], c2, kShifts ? add - off : add, kShifts ? add - off : add);
                        by = 1.f;
                        add = 0.f;
                    } else if constexpr (kShifts) {
                        add -= off;
                    }
                    if (wait_bias) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars.b_empty[buf]);
                    }
                    // a block needs masks unless all its pairs are visible (set after
                    // the bias, whose entries for unseen distances may hold anything)
                    const bool all = key0 + 63 <= first && (first + 127 - key0 < p.s.window || key0 + 63 < p.s.sinks);
                    if (!all) {
                        const int up = i - key0 + 1, down = i - p.s.window + 1 - key0, sk = p.s.sinks - key0;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t seen =
                                bits_below(up - 32 * h) & (~bits_below(down - 32 * h) | bits_below(sk - 32 * h));
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(seen >> c & 1)) x[32 * h + c] = -INFINITY;
                        }
                    }
                    float u[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) u[c] = max3(x[c], x[c + 8], x[c + 16]);
#pragma unroll
                    for (int c = 24; c < 56; c += 16)
#pragma unroll
                        for (int e = 0; e < 8; ++e) u[e] = max3(u[e], x[c + e], x[c + 8 + e]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[e] = fmaxf(u[e], x[56 + e]);
                    const float most = fmaxf(max3(max3(u[0], u[1], u[2]), u[3], u[4]), max3(u[5], u[6], u[7]));
                    const float top = fmaf(most, by, add);
                    if (__any_sync(0xffffffffu, top > m + kLazy || m == -INFINITY)) {
                        const float to = fmaxf(m, top);
                        const float keep = to == -INFINITY ? 1.f : ex2(m - to);
                        m = to;
                        l0 *= keep;
                        l1 *= keep;
                        if (n > 0) {
                            ok = mbar_wait_tight(&bars.o_done, (last + n - 1) & 1);
                            if (!__all_sync(0xffffffffu, ok)) {
                                ok = false;
                                break;
                            }
                            tcgen05_after_sync();
                            for (int c = 0; c < DP; c += 16) {
                                float o[16];
                                tmem_ld16(t_o + lanes + c, o);
#pragma unroll
                                for (int e = 0; e < 16; e += 2) mul2(o[e], o[e + 1], keep, keep);
                                tmem_st16(t_o + lanes + c, reinterpret_cast<const uint32_t*>(o));
                            }
                        }
                    }
                    // (nothing seen yet: all of the row's logits so far are -inf, the
                    // raw products may be finite where one bias hides the block)
                    const float less = m == -INFINITY ? -INFINITY : add - m;
#pragma unroll
                    for (int h = 0; h < 64; h += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int c = h; c < h + 32; c += 2) {
                            fma2(x[c], x[c + 1], by, less, less);
                            x[c] = ex2(x[c]);
                            x[c + 1] = ex2(x[c + 1]);
                            add2(l0, l1, x[c], x[c + 1]);
                            pk[(c - h) / 2] = pack2<DT>(x[c], x[c + 1]);
                        }
                        tmem_st16(t_s + h / 2, pk);
                    }
                    tmem_wait_st();
                    tcgen05_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.p_full[buf]);
                }
            };
            if (__any_sync(0xffffffffu, off != 0.f))
                walk(std::true_type{});
            else
                walk(std::false_type{});
            // ---- out = O / l, through the warp's rows of Q's tile
            // (a barrier of its own: o_done may be any of three phases along by now)
            if (ok) ok = mbar_wait_tight(&bars.o_last, turn & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
                tcgen05_after_sync();
                const float l = l0 + l1;
                const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing is zero
                unsigned char* qt = smem + L::q + turn % L::kQs * L::kQ;
#pragma unroll
                for (int c = 0; c < DP; c += 32) tmem_to_tile<DT>(qt, t_o + lanes, c, row, inv);
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.o_free);
                if (i < t.it.len) p.lse[(int64_t)t.head * p.N + t.it.start + i] = off + (m + log2f(l));
                store_tile_rows<DP>(p.out, qt, warp * 32, t.it.start, first, t.it.len, p.s.H, t.head, D, lane);
                fence_proxy_async_smem();  // before the next queries land here
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.q_empty[turn % L::kQs]);
            }
            g += steps;
            last += steps - 1;
            ++turn;
            // (a warp whose wait ran out waits for nothing any more, but meets the
            // others at the table's barriers to the last turn)
        } while (more());
    }
    if (!ok) atomicOr(p.s.error, ERR_TIMEOUT);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == 4) tmem_dealloc(tmem, L::cols);
}

template <int DT, int DP>
cudaError_t launch(const AttnForward& p, const AttnMaps& maps, cudaStream_t s) {
    const int64_t turns = p.max_items * p.s.H;
    if (p.ctas > 0 && p.ctas < turns)
        attn_fwd_mma_kernel<DT, DP, true><<<(unsigned)p.ctas, kThreads, Fwd<DP>::bytes, s>>>(p, maps);
    else
        attn_fwd_mma_kernel<DT, DP, false><<<(unsigned)turns, kThreads, Fwd<DP>::bytes, s>>>(p, maps);
    return cudaGetLastError();
}

template <int DT, int DP>
cudaError_t configure() {
    const cudaError_t e = cudaFuncSetAttribute(attn_fwd_mma_kernel<DT, DP, true>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, Fwd<DP>::bytes);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(attn_fwd_mma_kernel<DT, DP, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Fwd<DP>::bytes);
}

}  // namespace

cudaError_t attn_forward_mma_configure() {
    cudaError_t e = configure<DT_F16, 64>();
    if (e == cudaSuccess) e = configure<DT_F16, 128>();
    if (e == cudaSuccess) e = configure<DT_BF16, 64>();
    if (e == cudaSuccess) e = configure<DT_BF16, 128>();
    return e;
}

cudaError_t launch_attn_forward_mma(const AttnForward& p, const AttnMaps& maps, cudaStream_t s) {
    if (p.s.dtype == DT_F16) return p.s.D <= 64 ? launch<DT_F16, 64>(p, maps, s) : launch<DT_F16, 128>(p, maps, s);
    return p.s.D <= 64 ? launch<DT_BF16, 64>(p, maps, s) : launch<DT_BF16, 128>(p, maps, s);
}

}  // namespace tbe
