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
// The weights are rounded to the 16-bit type for the second product (the
// tensor cores' operand type); their sum is kept unrounded in fp32.
#include "attention_mma.cuh"

namespace tbe {

namespace {

constexpr int kThreads = 256;
constexpr float kLazy = 8.f;

template <int DP>
struct Fwd {
    static constexpr int kStages = DP == 64 ? 4 : 2;
    static constexpr int kTile = 64 * DP * 2;  // bytes of a K or V tile
    static constexpr int kQ = 128 * DP * 2;
    static constexpr int q = 0, k = kQ, v = k + kStages * kTile, bias = v + kStages * kTile;
    static constexpr int bytes = bias + kWholeEntries * 4 + 1024;  // 1024: the swizzle's alignment
    static constexpr int cols = 256;
};

struct FwdBars {
    uint64_t q_full, fix[2], k_full[4], k_empty[4], v_full[4], v_empty[4], s_full[2], p_full[2], o_done, o_last, b_full[2], b_empty[2];
};

template <int DT, int DP>
__global__ void __launch_bounds__(kThreads, 2) attn_fwd_mma_kernel(const AttnForward p, const __grid_constant__ AttnMaps maps) {
    using L = Fwd<DP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ FwdBars bars;
    __shared__ uint32_t tmem_slot;
    __shared__ float uniform_bias[2];
    __shared__ int is_uniform[2];

    const int64_t w = blockIdx.x / p.s.H;
    const int head = (int)(blockIdx.x % p.s.H);
    AttnItem it;
    if (!find_item(p.src, w, it)) return;
    const int kvh = head / p.s.G, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int first = it.tile * 128, D = p.s.D;
    const int ksteps = (D + 15) / 16;
    // visible key blocks: [0, sink_blocks) and [lo, hi)
    const int hi = tmin(first + 127, it.len - 1) / 64 + 1;
    const int64_t from = (int64_t)first - p.s.window + 1;
    const int lo = from > 0 ? (int)(from / 64) : 0;
    const int sink_blocks = tmin((p.s.sinks + 63) / 64, lo);
    const int steps = sink_blocks + hi - lo;
    auto block_of = [&](int n) { return n < sink_blocks ? n : lo + n - sink_blocks; };

    const uint32_t sbase = smem_u32(smem);
    if (threadIdx.x == 0) {
        mbar_init(&bars.q_full, 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars.k_full[i], 1);
            mbar_init(&bars.k_empty[i], 1);
            mbar_init(&bars.v_full[i], 1);
            mbar_init(&bars.v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i], 4);
            mbar_init(&bars.b_full[i], 1);
            mbar_init(&bars.b_empty[i], 4);
        }
        mbar_init(&bars.o_done, 1);
        mbar_init(&bars.fix[0], 1);
        mbar_init(&bars.fix[1], 1);
        mbar_init(&bars.o_last, 1);
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
    float last_bias;
    const bool whole = keep_whole<DT>(p.s, p.bias, head, last_bias);
    if (warp == 5 || warp == 6) {
        // ---- loaders: warp 5 Q and K, warp 6 V
        uint32_t fix_phase = 0;
        auto place = [&](int n) { return make_int2(block_of(n) * 64, kvh); };
        if (warp == 5)
            ok = load_tile<128, DP>(smem + L::q, maps.q, it, head, first, &bars.q_full, &bars.fix[0], fix_phase, lane) &&
                 load_ring<DP, L::kStages>(smem + L::k, maps.k, it, bars.k_full, bars.k_empty, &bars.fix[0], fix_phase,
                                           steps, lane, place);
        else
            ok = load_ring<DP, L::kStages>(smem + L::v, maps.v, it, bars.v_full, bars.v_empty, &bars.fix[1], fix_phase,
                                           steps, lane, place);
    } else if (warp == 7) {
        // ---- bias by distance: entry x of the block's table is the bias at
        // distance base + x - 63, x in [0, 191)
        if (p.bias && !whole) {
            float* bt = reinterpret_cast<float*>(smem + L::bias);
            for (int n = 0; n < steps && ok; ++n) {
                const int buf = n & 1;
                if (n >= 2) ok = mbar_wait_tight(&bars.b_empty[buf], ((n / 2) - 1) & 1);
                if (!ok) break;
                const int base = first - block_of(n) * 64;
                const int least = tmax(0, base - 63), most = base + 127;
                const int b0 = attn_bucket(p.s, least), b1 = attn_bucket(p.s, tmax(most, 0));
                const float same = bias_base2(load_elem<DT>(p.bias, (int64_t)b0 * p.s.H + head));
                // a bias that swallows the logits (a type's lowest value) does
                // so in the table's addition only
                const bool one = b0 == b1 && (same > -1e30f || same == -INFINITY);
                if (lane == 0) {
                    is_uniform[buf] = one;
                    uniform_bias[buf] = same;
                }
                if (!one)
                    for (int x = lane; x < 191; x += 32) {
                        const int d = base + x - 63;
                        bt[buf * 192 + x] =
                            d >= 0 ? bias_base2(load_elem<DT>(p.bias, (int64_t)attn_bucket(p.s, d) * p.s.H + head))
                                   : 0.f;
                    }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.b_full[buf]);
            }
        }
    } else if (warp == 4) {
        // ---- products
        const uint32_t id_s = mma_idesc(DT == DT_BF16, 128, 64);
        const uint32_t id_o = mma_idesc(DT == DT_BF16, 128, ksteps * 16) | kMnMajorB;
        const uint64_t dq = smem_desc_sw128(sbase + L::q, 1024), dk = smem_desc_sw128(sbase + L::k, 1024);
        const uint64_t dv = smem_desc_mn(sbase + L::v, 64 * 128);
        ok = mbar_wait_tight(&bars.q_full, 0);
        auto scores = [&](int n) {
            const int st = n % L::kStages;
            const bool in = mbar_wait_tight(&bars.k_full[st], (n / L::kStages) & 1);
            if (!__all_sync(0xffffffffu, in)) return false;
            tcgen05_after_sync();
            if (elect_one()) {
                issue_scores<DP>(tmem + (n & 1) * 64, dq, dk + st * (L::kTile / 16), id_s, ksteps);
                if (n + L::kStages < steps) mma_commit(&bars.k_empty[st]);
                mma_commit(&bars.s_full[n & 1]);
            }
            __syncwarp();
            return true;
        };
        ok = __all_sync(0xffffffffu, ok) && scores(0);
        if (ok && steps > 1) ok = scores(1);
        for (int n = 0; n < steps && ok; ++n) {
            const int st = n % L::kStages;
            ok = mbar_wait_tight(&bars.v_full[st], (n / L::kStages) & 1) &&
                 mbar_wait_tight(&bars.p_full[n & 1], (n / 2) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tcgen05_after_sync();
            if (elect_one()) {
                issue_product(t_o, tmem + (n & 1) * 64, dv + st * (L::kTile / 16), id_o, n > 0);
                if (n + L::kStages < steps) mma_commit(&bars.v_empty[st]);
                mma_commit(n + 1 < steps ? &bars.o_done : &bars.o_last);
            }
            __syncwarp();
            if (n + 2 < steps) {
                // block n + 2's scores overwrite P(n): wait for its product
                ok = mbar_wait_tight(&bars.o_done, n & 1);
                ok = __all_sync(0xffffffffu, ok) && scores(n + 2);
            }
        }
    } else {
        // ---- softmax: thread = query
        const int row = threadIdx.x, i = first + row;
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const float c2 = p.s.scale * kLog2e;
        const float* bt = reinterpret_cast<const float*>(smem + L::bias);
        if (p.bias && whole) {
            fill_bias<DT>(reinterpret_cast<float*>(smem + L::bias), p.s, p.bias, head, first + 127, row, 128);
            asm volatile("bar.sync 1, 128;" ::: "memory");
        }
        const bool wait_bias = p.bias && !whole;
        float m = -INFINITY, l0 = 0.f, l1 = 0.f;
        for (int n = 0; n < steps; ++n) {
            const int buf = n & 1;
            const uint32_t t_s = tmem + buf * 64 + lanes;
            ok = mbar_wait_tight(&bars.s_full[buf], (n / 2) & 1);
            if (ok && wait_bias) ok = mbar_wait_tight(&bars.b_full[buf], (n / 2) & 1);
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
            const int key0 = block_of(n) * 64;
            const bool table = p.bias && (whole ? first - key0 - 63 < p.s.far : !is_uniform[buf]);
            // a block needs masks unless all its pairs are visible
            const bool all = key0 + 63 <= first && (first + 127 - key0 < p.s.window || key0 + 63 < p.s.sinks);
            if (!all) {
                const int up = i - key0 + 1, down = i - p.s.window + 1 - key0, sk = p.s.sinks - key0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t seen = bits_below(up - 32 * h) & (~bits_below(down - 32 * h) | bits_below(sk - 32 * h));
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!(seen >> c & 1)) x[32 * h + c] = -INFINITY;
                }
            }
            // logit = x * by + add: with a table it is formed here, else (one
            // bias for the block, and c2 > 0) the maximum is taken of the raw
            // products and one multiply-add before ex2 does it all
            float by = c2, add = wait_bias ? uniform_bias[buf] : last_bias;
            if (table) {
                const float* b = bt + (whole ? i - key0 + 127 : buf * 192 + row + 63);
#pragma unroll
                for (int c = 0; c < 64; c += 2) fma2(x[c], x[c + 1], c2, b[-c], b[-c - 1]);
                by = 1.f;
                add = 0.f;
            }
            if (wait_bias) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.b_empty[buf]);
            }
            float t[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) t[c] = max3(x[c], x[c + 8], x[c + 16]);
#pragma unroll
            for (int c = 24; c < 56; c += 16)
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = max3(t[e], x[c + e], x[c + 8 + e]);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = fmaxf(t[e], x[56 + e]);
            const float top = fmaf(fmaxf(max3(max3(t[0], t[1], t[2]), t[3], t[4]), max3(t[5], t[6], t[7])), by, add);
            if (__any_sync(0xffffffffu, top > m + kLazy || m == -INFINITY)) {
                const float to = fmaxf(m, top);
                const float keep = to == -INFINITY ? 1.f : ex2(m - to);
                m = to;
                l0 *= keep;
                l1 *= keep;
                if (n > 0) {
                    ok = mbar_wait_tight(&bars.o_done, (n - 1) & 1);
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
            const float less = m == -INFINITY ? 0.f : add - m;
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
        // ---- out = O / l, through the warp's rows of Q's tile
        // (a barrier of its own: o_done may be any of three phases along by now)
        if (ok) ok = mbar_wait_tight(&bars.o_last, 0);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
            tcgen05_after_sync();
            const float l = l0 + l1;
            const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing is zero
            unsigned char* qt = smem + L::q;
#pragma unroll
            for (int c = 0; c < DP; c += 32) tmem_to_tile<DT>(qt, t_o + lanes, c, row, inv);
            if (i < it.len) p.lse[(int64_t)head * p.N + it.start + i] = m + log2f(l);
            __syncwarp();
            store_tile_rows<DP>(p.out, qt, warp * 32, it.start, first, it.len, p.s.H, head, D, lane);
        }
    }
    if (!ok) atomicOr(p.s.error, ERR_TIMEOUT);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == 4) tmem_dealloc(tmem, L::cols);
}

template <int DT, int DP>
cudaError_t launch(const AttnForward& p, const AttnMaps& maps, int64_t max_items, cudaStream_t s) {
    attn_fwd_mma_kernel<DT, DP><<<(unsigned)(max_items * p.s.H), kThreads, Fwd<DP>::bytes, s>>>(p, maps);
    return cudaGetLastError();
}

template <int DT, int DP>
cudaError_t configure() {
    return cudaFuncSetAttribute(attn_fwd_mma_kernel<DT, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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

cudaError_t launch_attn_forward_mma(const AttnForward& p, const AttnMaps& maps, int64_t max_items, cudaStream_t s) {
    if (p.s.dtype == DT_F16) return p.s.D <= 64 ? launch<DT_F16, 64>(p, maps, max_items, s) : launch<DT_F16, 128>(p, maps, max_items, s);
    return p.s.D <= 64 ? launch<DT_BF16, 64>(p, maps, max_items, s) : launch<DT_BF16, 128>(p, maps, max_items, s);
}

}  // namespace tbe
