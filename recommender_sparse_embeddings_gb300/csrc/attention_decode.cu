// The serving form: new tokens' keys and values go to a paged cache, and one
// new token per history attends to its cache.
//
// The cache of history b is the pages table[b][0], table[b][1], ...; token j
// is row j % page of page table[b][j / page].  Only the visible rows are
// read: the first `sinks` and the newest `window`.  What a page holds beyond
// a history's length is never loaded, whatever its bits are.
#include "attention.cuh"

namespace tbe {

namespace {

constexpr int kAppendThreads = 256;

// One warp per new token: finds its history by bisection of the offsets,
// then copies the token's key and value rows into its page.
template <typename I>
__global__ void __launch_bounds__(kAppendThreads) attn_append_kernel(const AttnAppend p) {
    const int64_t t = (int64_t)blockIdx.x * (kAppendThreads / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (t >= p.N) return;
    const I* off = static_cast<const I*>(p.offsets);
    int lo = 0, hi = p.B - 1;  // the last history that starts at or before t
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if ((int64_t)off[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int64_t from = (int64_t)off[lo], to = (int64_t)off[lo + 1];
    if (from < 0 || t < from || t >= to) {
        if (lane == 0) atomicOr(p.error, ERR_OFFSETS);
        return;
    }
    const int64_t pos = (int64_t)p.before[lo] + (t - from);
    if (p.before[lo] < 0 || pos >= (int64_t)p.width * p.page.n) {
        if (lane == 0) atomicOr(p.error, ERR_OOB);
        return;
    }
    const uint32_t pg = fast_div((uint32_t)pos, p.page);
    const int row = (int)((uint32_t)pos - pg * p.page.n);
    const int32_t page = p.table[(int64_t)lo * p.width + pg];
    if (page < 0 || page >= p.num_pages) {
        if (lane == 0) atomicOr(p.error, ERR_OOB);
        return;
    }
    const char* ks = static_cast<const char*>(p.k.data) + t * p.k.token_stride * p.e;
    const char* vs = static_cast<const char*>(p.v.data) + t * p.v.token_stride * p.e;
    char* kd = static_cast<char*>(p.kp) + (page * p.k_page + row * p.k_token) * p.e;
    char* vd = static_cast<char*>(p.vp) + (page * p.v_page + row * p.v_token) * p.e;
    const int bytes = p.D * p.e, unit = p.vec ? 16 : p.e, per = bytes / unit;
    for (int c = lane; c < p.Hk * per; c += 32) {
        const int h = c / per, x = c % per * unit;
        const char* a = ks + h * p.k.head_stride * p.e + x;
        const char* b = vs + h * p.v.head_stride * p.e + x;
        char* ka = kd + h * p.k_head * p.e + x;
        char* vb = vd + h * p.v_head * p.e + x;
        if (p.vec) {
            *reinterpret_cast<uint4*>(ka) = __ldg(reinterpret_cast<const uint4*>(a));
            *reinterpret_cast<uint4*>(vb) = __ldg(reinterpret_cast<const uint4*>(b));
        } else if (p.e == 4) {
            *reinterpret_cast<uint32_t*>(ka) = __ldg(reinterpret_cast<const uint32_t*>(a));
            *reinterpret_cast<uint32_t*>(vb) = __ldg(reinterpret_cast<const uint32_t*>(b));
        } else {
            *reinterpret_cast<uint16_t*>(ka) = __ldg(reinterpret_cast<const uint16_t*>(a));
            *reinterpret_cast<uint16_t*>(vb) = __ldg(reinterpret_cast<const uint16_t*>(b));
        }
    }
}

constexpr int kWarps = 4;

// The visible rows of a cache of len tokens, as one range [0, sinks + len - lo):
// index x is token x below `sinks` and token lo + x - sinks from there on.
struct Visible {
    int sinks, lo, count;
};

__device__ __forceinline__ Visible visible_rows(const AttnShape& s, int len) {
    const int lo = len > s.window ? len - s.window : 0;
    const int sinks = tmin(s.sinks, lo);
    return Visible{sinks, lo, sinks + len - lo};
}

__device__ __forceinline__ int cache_length(const AttnDecode& p, int b) {
    const int len = __ldg(p.lengths + b);
    return len < 0 || (int64_t)len > p.max_length ? -1 : len;
}

// The buckets' biases of the CTA's heads, table[head][bucket] in base 2, a warp
// per head.  Where a head has one of large magnitude the largest that its new
// token sees is taken off them: fp32 holds no logit beside it.  (All CTAs of a
// history take off the same, so their shares still join.)
template <int DT, int HEADS, int WARPS>
__device__ __forceinline__ void load_biases(float* table, const AttnShape& s, const void* bias, int head0, int heads,
                                            int len) {
    const int lane = threadIdx.x % 32;
#pragma unroll 1
    for (int h = threadIdx.x / 32; h < HEADS; h += WARPS) {
        auto bias_of = [&](int b) {
            return h < heads ? bias_base2(load_elem<DT>(bias, (int64_t)b * s.H + head0 + h)) : 0.f;
        };
        bool large = false;
#pragma unroll 1
        for (int b = lane; b < s.buckets; b += 32) {
            const float x = bias_of(b);
            table[h * s.buckets + b] = x;
            large |= attn_coarse(x);
        }
        if (__any_sync(0xffffffffu, large) && len > 0) {
            float top = attn_bias_top(s, len - 1, lane, 32, bias_of);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float off = attn_bias_off(top);
#pragma unroll 1
            for (int b = lane; b < s.buckets; b += 32) table[h * s.buckets + b] = bias_of(b) - off;
        }
    }
    __syncthreads();
}

// The 16-byte vectors that a lane holds of a row; columns from D on keep what
// the registers hold (zeros, from the start).
template <int DT, int NV>
__device__ __forceinline__ void load_vecs(uint4 (&u)[NV], const typename Elem<DT>::type* row, int col, int step, int D,
                                          int vec) {
    using E = typename Elem<DT>::type;
    constexpr int V = 16 / sizeof(E);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int c = col + n * step;
        if (vec) {
            if (c < D) u[n] = __ldg(reinterpret_cast<const uint4*>(row + c));
        } else {
            E e[V];
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = c + i < D ? row[c + i] : E(0.f);
            u[n] = *reinterpret_cast<uint4*>(e);
        }
    }
}

// One CTA: `chunk` visible rows of one history for GT query heads of one
// key-value head.  LPR lanes hold one row (16 bytes each, NV times); each
// such group of lanes runs its own softmax over its rows, U rows a step, and
// the groups are joined at the end.
template <int DT, int GT, int LPR, int NV>
__global__ void __launch_bounds__(kWarps * 32) attn_decode_kernel(const AttnDecode p) {
    using E = typename Elem<DT>::type;
    constexpr int V = 16 / sizeof(E), RPW = 32 / LPR, U = GT > 4 ? 2 : 4, STEP = kWarps * RPW * U;
    constexpr int W = V * NV;
    extern __shared__ float dsm[];
    __shared__ float stat[kWarps][GT][2];
    const int hchunks = (p.s.G + GT - 1) / GT;
    uint32_t x = blockIdx.x;
    const int split = (int)(x % p.splits);
    x /= p.splits;
    const int hc = (int)(x % hchunks);
    x /= hchunks;
    const int kvh = (int)(x % p.s.Hk), b = (int)(x / p.s.Hk);
    const int g0 = hc * GT, gn = tmin(GT, p.s.G - g0), head0 = kvh * p.s.G + g0;
    const int len = cache_length(p, b);
    if (len < 0 && threadIdx.x == 0 && split == 0) atomicOr(p.s.error, ERR_OOB);
    const Visible vis = visible_rows(p.s, tmax(len, 0));
    if (split > 0 && split * p.chunk >= vis.count) return;
    const int begin = split * p.chunk, end = vis.count - begin <= p.chunk ? vis.count : begin + p.chunk;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = lane / LPR;
    const int col = lane % LPR * V;
    constexpr int cstep = LPR * V;
    const float c2 = p.s.scale * kLog2e;

    if (p.bias) load_biases<DT, GT, kWarps>(dsm, p.s, p.bias, head0, gn, len);
    float q[GT][W], o[GT][W], m[GT], l[GT];
#pragma unroll
    for (int g = 0; g < GT; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
        uint4 u[NV];
#pragma unroll
        for (int n = 0; n < NV; ++n) u[n] = make_uint4(0, 0, 0, 0);
        if (g < gn) {
            const E* row = static_cast<const E*>(p.q.data) + b * p.q.token_stride + (head0 + g) * p.q.head_stride;
            load_vecs<DT, NV>(u, row, col, cstep, p.s.D, p.vec);
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) unpack16<DT>(u[n], &q[g][n * V]);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            q[g][i] *= c2;
            o[g][i] = 0.f;
        }
    }
    const E* kbase = static_cast<const E*>(p.kp) + kvh * p.k_head;
    const E* vbase = static_cast<const E*>(p.vp) + kvh * p.v_head;
    const int32_t* table = p.table + (int64_t)b * p.width;

    // Where the lane's rows of a step lie (elements from the bases) and how far
    // they are from the new token; -1 for a row that is not there.  Such a row
    // leaves its registers as they are: its logit is replaced, its weight is 0.
    struct Place {
        int64_t k[U], v[U];
        int dist[U];
    };
    auto find = [&](int x0) {
        Place at;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int xi = x0 + (u * kWarps + warp) * RPW + sub;
            const int j = xi < vis.sinks ? xi : vis.lo + xi - vis.sinks;
            at.dist[u] = -1;
            at.k[u] = at.v[u] = 0;
            if (xi < end) {
                const uint32_t pg = fast_div((uint32_t)j, p.page);
                const int row = (int)((uint32_t)j - pg * p.page.n);
                const int32_t page = __ldg(table + pg);
                if (page >= 0 && page < p.num_pages) {
                    at.dist[u] = len - 1 - j;
                    at.k[u] = page * p.k_page + row * p.k_token;
                    at.v[u] = page * p.v_page + row * p.v_token;
                } else {
                    atomicOr(p.s.error, ERR_OOB);
                }
            }
        }
        return at;
    };
    uint4 kr[U][NV], vr[U][NV];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int n = 0; n < NV; ++n) kr[u][n] = vr[u][n] = make_uint4(0, 0, 0, 0);
    auto load_keys = [&](const Place& at) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (at.dist[u] >= 0) load_vecs<DT, NV>(kr[u], kbase + at.k[u], col, cstep, p.s.D, p.vec);
    };
    auto load_values = [&](const Place& at) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (at.dist[u] >= 0) load_vecs<DT, NV>(vr[u], vbase + at.v[u], col, cstep, p.s.D, p.vec);
    };
    // the next step's keys are fetched before this step's softmax, its values
    // after this step's product
    Place here = find(begin), next = find(begin + STEP);
    load_keys(here);
    load_values(here);
    for (int x0 = begin; x0 < end; x0 += STEP) {
        float s[U][GT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[W];
#pragma unroll
            for (int n = 0; n < NV; ++n) unpack16<DT>(kr[u][n], &f[n * V]);
#pragma unroll
            for (int g = 0; g < GT; ++g) {
                float t = 0.f;
#pragma unroll
                for (int i = 0; i < W; ++i) t = fmaf(q[g][i], f[i], t);
#pragma unroll
                for (int w = LPR / 2; w > 0; w >>= 1) t += __shfl_xor_sync(0xffffffffu, t, w);
                s[u][g] = t;
            }
            if (p.bias) {
                const int bk = here.dist[u] >= 0 ? attn_bucket(p.s, here.dist[u]) : 0;
#pragma unroll
                for (int g = 0; g < GT; ++g) s[u][g] += dsm[g * p.s.buckets + bk];
            }
        }
        load_keys(next);
#pragma unroll
        for (int g = 0; g < GT; ++g) {
            float top = m[g];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (here.dist[u] < 0) s[u][g] = -INFINITY;
                top = fmaxf(top, s[u][g]);
            }
            const float safe = top == -INFINITY ? 0.f : top;
            const float keep = ex2(m[g] - safe);
            m[g] = top;
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u][g] = ex2(s[u][g] - safe);
                sum += s[u][g];
            }
            l[g] = l[g] * keep + sum;
#pragma unroll
            for (int i = 0; i < W; ++i) o[g][i] *= keep;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[W];
#pragma unroll
            for (int n = 0; n < NV; ++n) unpack16<DT>(vr[u][n], &f[n * V]);
#pragma unroll
            for (int g = 0; g < GT; ++g)
#pragma unroll
                for (int i = 0; i < W; ++i) o[g][i] = fmaf(s[u][g], f[i], o[g][i]);
        }
        load_values(next);
        here = next;
        next = find(x0 + 2 * STEP);
    }
    // join the warp's groups, then the CTA's warps
    float* osm = dsm + (p.bias ? GT * p.s.buckets : 0);  // [kWarps][GT][LPR * W]
#pragma unroll
    for (int g = 0; g < GT; ++g) {
        float top = m[g];
#pragma unroll
        for (int w = LPR; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        const float keep = ex2(m[g] - (top == -INFINITY ? 0.f : top));
        float sum = l[g] * keep;
#pragma unroll
        for (int w = LPR; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float t = o[g][i] * keep;
#pragma unroll
            for (int w = LPR; w < 32; w <<= 1) t += __shfl_xor_sync(0xffffffffu, t, w);
            if (sub == 0) osm[(warp * GT + g) * (LPR * W) + col + (i / V) * cstep + i % V] = t;
        }
        if (lane == 0) {
            stat[warp][g][0] = top;
            stat[warp][g][1] = sum;
        }
    }
    __syncthreads();
    const bool whole = vis.count <= p.chunk;
    for (int i = threadIdx.x; i < gn * p.s.D; i += kWarps * 32) {
        const int g = i / p.s.D, d = i % p.s.D;
        float top = -INFINITY, sum = 0.f, t = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[w][g][0]);
        const float safe = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float keep = ex2(stat[w][g][0] - safe);
            sum += stat[w][g][1] * keep;
            t += osm[(w * GT + g) * (LPR * W) + d] * keep;
        }
        const int64_t row = (int64_t)b * p.s.H + head0 + g;
        if (whole) {
            store_elem<DT>(p.out, row * p.s.D + d, sum == 0.f ? 0.f : t / sum);  // an empty cache gives zeros
        } else {
            float* to = p.part + (row * p.splits + split) * (p.s.D + 2);
            to[d] = t;
            if (d == 0) {
                to[p.s.D] = top;
                to[p.s.D + 1] = sum;
            }
        }
    }
}

// ---- 16-bit caches: the products on mma.sync (m16n8k16).  One new token is a
// row of G heads against the cache, far from a tcgen05 tile, and the work is
// bound by the cache's bytes: on the FMA units the dot products and their
// shuffles took about 140 instructions a kilobyte of cache (405 us for 128
// histories of 4000 rows of 4 x 128, twice the bytes' time); with a warp's
// tensor instruction it is about 15.
//
// A warp takes 16 rows a step.  Lane (g, t) = (lane / 4, lane % 4).
//   S [heads x rows] = Q K^T: a lane holds 16-byte chunks t, t + 4, .. of rows
//     g and g + 8 as they lie in memory.  The product runs over all columns, so
//     which k slot a column takes does not matter as long as Q's fragment says
//     the same: a chunk is two instructions' operand as loaded.
//   O^T [columns x heads] = V^T P^T: a lane holds chunk g (g + 8) of rows 2t,
//     2t + 1, 2t + 8, 2t + 9; a byte permute pairs neighbouring rows, and S's
//     accumulator is P^T's fragment as it stands.
// The next step's keys are fetched before this step's softmax, its values after
// this step's product: a warp keeps 8 KB in flight (head_dim 128).

constexpr int kMmaHeads = 8;
constexpr int kMmaWarps = 4;

template <int DT>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    if constexpr (DT == DT_BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int DT>
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
    uint32_t r;
    if constexpr (DT == DT_BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int DT, int DP>
__global__ void __launch_bounds__(kMmaWarps * 32) __maxnreg__(DP == 64 ? 96 : 168)
    attn_decode_mma_kernel(const AttnDecode p) {
    constexpr int KC = DP / 32, VC = DP / 64;  // 16-byte chunks a lane holds of a key row, of a value row
    constexpr int STEP = kMmaWarps * 16;
    extern __shared__ float dsm[];  // bias by bucket [8][buckets]; then the warps' sums [warps][8][DP]
    __shared__ float stat[kMmaWarps][kMmaHeads][2];
    const int hchunks = (p.s.G + kMmaHeads - 1) / kMmaHeads;
    uint32_t bx = blockIdx.x;
    const int split = (int)(bx % p.splits);
    bx /= p.splits;
    const int hc = (int)(bx % hchunks);
    bx /= hchunks;
    const int kvh = (int)(bx % p.s.Hk), b = (int)(bx / p.s.Hk);
    const int g0 = hc * kMmaHeads, gn = tmin(kMmaHeads, p.s.G - g0), head0 = kvh * p.s.G + g0;
    const int len = cache_length(p, b);
    if (len < 0 && threadIdx.x == 0 && split == 0) atomicOr(p.s.error, ERR_OOB);
    const Visible vis = visible_rows(p.s, tmax(len, 0));
    if (split > 0 && split * p.chunk >= vis.count) return;
    const int begin = split * p.chunk, end = vis.count - begin <= p.chunk ? vis.count : begin + p.chunk;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int D = p.s.D;
    if (p.bias) load_biases<DT, kMmaHeads, kMmaWarps>(dsm, p.s, p.bias, head0, gn, len);
    const float* bias = dsm + g * p.s.buckets;
    const float c2 = p.s.scale * kLog2e;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 q[KC];
#pragma unroll
    for (int c = 0; c < KC; ++c) {
        const int col = (t + 4 * c) * 8;
        q[c] = zero;
        if (g < gn && col < D)
            q[c] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q.data) +
                                                        b * p.q.token_stride + (head0 + g) * p.q.head_stride + col));
    }
    const uint16_t* kbase = static_cast<const uint16_t*>(p.kp) + kvh * p.k_head;
    const uint16_t* vbase = static_cast<const uint16_t*>(p.vp) + kvh * p.v_head;
    const int32_t* table = p.table + (int64_t)b * p.width;

    auto row_of = [&](int x) { return x < vis.sinks ? x : vis.lo + x - vis.sinks; };
    const float last_bias = p.bias ? bias[p.s.buckets - 1] : 0.f;
    // lanes 0-15: where the keys of the step's 16 rows lie, lanes 16-31 the
    // values (elements from the base); -1 for none
    auto find = [&](int x0) {
        const int xi = x0 + lane % 16;
        if (xi >= end) return (int64_t)-1;
        const int j = row_of(xi);
        const uint32_t pg = fast_div((uint32_t)j, p.page);
        const int row = (int)((uint32_t)j - pg * p.page.n);
        const int32_t page = __ldg(table + pg);
        if (page < 0 || page >= p.num_pages) {
            atomicOr(p.s.error, ERR_OOB);
            return (int64_t)-1;
        }
        return lane < 16 ? page * p.k_page + row * p.k_token : page * p.v_page + row * p.v_token;
    };
    // A row that is not there leaves its registers as they are: zeros or an
    // earlier row of this history.  Its logit is replaced, its weight is 0.
    uint4 kr[2][KC], vr[4][VC];
#pragma unroll
    for (int c = 0; c < KC; ++c) kr[0][c] = kr[1][c] = zero;
#pragma unroll
    for (int c = 0; c < VC; ++c) vr[0][c] = vr[1][c] = vr[2][c] = vr[3][c] = zero;
    auto load_keys = [&](int64_t where) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int64_t at = __shfl_sync(0xffffffffu, where, g + 8 * r);
            const uint4* row = reinterpret_cast<const uint4*>(kbase + at + t * 8);
#pragma unroll
            for (int c = 0; c < KC; ++c)
                if (at >= 0 && (t + 4 * c) * 8 < D) kr[r][c] = __ldg(row + 4 * c);
        }
    };
    auto load_values = [&](int64_t where) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t at = __shfl_sync(0xffffffffu, where, 16 + 2 * t + (r & 1) + 8 * (r >> 1));
            const uint4* row = reinterpret_cast<const uint4*>(vbase + at + g * 8);
#pragma unroll
            for (int c = 0; c < VC; ++c)
                if (at >= 0 && (g + 8 * c) * 8 < D) vr[r][c] = __ldg(row + 8 * c);
        }
    };

    float m = -INFINITY, l = 0.f;  // of head g (l: this lane's rows)
    float o[VC * 4][4];
#pragma unroll
    for (int i = 0; i < VC * 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    int x0 = begin + warp * 16;
    int64_t where = find(x0), next = find(x0 + STEP);
    load_keys(where);
    load_values(where);
    for (; x0 < end; x0 += STEP) {
        float s[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[r][e] = 0.f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                mma_16816<DT>(s[r], q[c].x, 0u, q[c].y, 0u, kr[r][c].x, kr[r][c].y);
                mma_16816<DT>(s[r], q[c].z, 0u, q[c].w, 0u, kr[r][c].z, kr[r][c].w);
            }
        }
        // rows 2t, 2t + 1, 2t + 8, 2t + 9 of the step, for head g; rows without
        // a page count as not there
        const uint32_t there = __ballot_sync(0xffffffffu, where >= 0);
        float y[4] = {s[0][0], s[0][1], s[1][0], s[1][1]};
        const int64_t now = next;
        load_keys(now);
        next = find(x0 + 2 * STEP);
        float top = m;
        // the step's last row is its nearest: from `far` on all share a bucket
        const bool distant = x0 + 15 < end && len - 1 - row_of(x0 + 15) >= p.s.far;
        float add[4] = {last_bias, last_bias, last_bias, last_bias};
        if (p.bias && !distant) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int xi = x0 + 2 * t + (e & 1) + 8 * (e >> 1);
                add[e] = bias[xi < end ? attn_bucket(p.s, len - 1 - row_of(xi)) : 0];
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e] = fmaf(y[e], c2, add[e]);
            if (!(there >> (2 * t + (e & 1) + 8 * (e >> 1)) & 1)) y[e] = -INFINITY;
            top = fmaxf(top, y[e]);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float safe = top == -INFINITY ? 0.f : top;
        if (__any_sync(0xffffffffu, top > m)) {
            const float keep = ex2(m - safe);
            l *= keep;
            const float k0 = __shfl_sync(0xffffffffu, keep, 8 * t), k1 = __shfl_sync(0xffffffffu, keep, 8 * t + 4);
#pragma unroll
            for (int i = 0; i < VC * 4; ++i) {
                o[i][0] *= k0;
                o[i][1] *= k1;
                o[i][2] *= k0;
                o[i][3] *= k1;
            }
            m = top;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e] = ex2(y[e] - safe);
            l += y[e];
        }
        const uint32_t p0 = round2<DT>(y[0], y[1]), p1 = round2<DT>(y[2], y[3]);
#pragma unroll
        for (int c = 0; c < VC; ++c) {
            const uint32_t* r0 = &vr[0][c].x;
            const uint32_t* r1 = &vr[1][c].x;
            const uint32_t* r2 = &vr[2][c].x;
            const uint32_t* r3 = &vr[3][c].x;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mma_16816<DT>(o[c * 4 + i], __byte_perm(r0[i], r1[i], 0x5410), __byte_perm(r0[i], r1[i], 0x7632),
                              __byte_perm(r2[i], r3[i], 0x5410), __byte_perm(r2[i], r3[i], 0x7632), p0, p1);
        }
        load_values(now);
        where = now;
    }
    // join the lanes of a head, then the CTA's warps
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (t == 0) {
        stat[warp][g][0] = m;
        stat[warp][g][1] = l;
    }
    float* osm = dsm + (p.bias ? kMmaHeads * p.s.buckets : 0);
#pragma unroll
    for (int c = 0; c < VC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                osm[(warp * kMmaHeads + 2 * t + (e & 1)) * DP + (g + 8 * c) * 8 + 2 * i + (e >> 1)] = o[c * 4 + i][e];
    __syncthreads();
    const bool whole = vis.count <= p.chunk;
    for (int i = threadIdx.x; i < gn * D; i += kMmaWarps * 32) {
        const int h = i / D, d = i % D;
        float top = -INFINITY, sum = 0.f, v = 0.f;
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) top = fmaxf(top, stat[w][h][0]);
        const float safe = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) {
            const float keep = ex2(stat[w][h][0] - safe);
            sum += stat[w][h][1] * keep;
            v += osm[(w * kMmaHeads + h) * DP + d] * keep;
        }
        const int64_t row = (int64_t)b * p.s.H + head0 + h;
        if (whole) {
            store_elem<DT>(p.out, row * D + d, sum == 0.f ? 0.f : v / sum);  // an empty cache gives zeros
        } else {
            float* to = p.part + (row * p.splits + split) * (D + 2);
            to[d] = v;
            if (d == 0) {
                to[D] = top;
                to[D + 1] = sum;
            }
        }
    }
}

// Joins the chunks of one history and head: the partial sums scaled to the
// largest of their maxima, added in the chunks' order.
template <int DT>
__global__ void __launch_bounds__(128) attn_decode_join_kernel(const AttnDecode p) {
    const int b = (int)(blockIdx.x / p.s.H);
    const int len = cache_length(p, b);
    const Visible vis = visible_rows(p.s, tmax(len, 0));
    if (vis.count <= p.chunk) return;  // written by its one CTA
    const int n = (vis.count + p.chunk - 1) / p.chunk;
    const float* part = p.part + (int64_t)blockIdx.x * p.splits * (p.s.D + 2);
    const int ld = p.s.D + 2;
    float top = -INFINITY;
    for (int i = 0; i < n; ++i) top = fmaxf(top, part[i * ld + p.s.D]);
    const float safe = top == -INFINITY ? 0.f : top;
    for (int d = threadIdx.x; d < p.s.D; d += 128) {
        float sum = 0.f, t = 0.f;
        for (int i = 0; i < n; ++i) {
            const float keep = ex2(part[i * ld + p.s.D] - safe);
            sum += part[i * ld + p.s.D + 1] * keep;
            t += part[i * ld + d] * keep;
        }
        store_elem<DT>(p.out, (int64_t)blockIdx.x * p.s.D + d, sum == 0.f ? 0.f : t / sum);
    }
}

template <int DT, int GT, int LPR, int NV>
cudaError_t decode(const AttnDecode& p, cudaStream_t s) {
    constexpr int W = 16 / sizeof(typename Elem<DT>::type) * NV;
    const int64_t grid = (int64_t)p.splits * ((p.s.G + GT - 1) / GT) * p.s.Hk * p.B;
    const size_t smem = sizeof(float) * ((p.bias ? (size_t)GT * p.s.buckets : 0) + (size_t)kWarps * GT * LPR * W);
    attn_decode_kernel<DT, GT, LPR, NV><<<(unsigned)grid, kWarps * 32, smem, s>>>(p);
    return cudaGetLastError();
}

template <int DT, int DP>
cudaError_t decode_mma(const AttnDecode& p, cudaStream_t s) {
    const int64_t grid = (int64_t)p.splits * ((p.s.G + kMmaHeads - 1) / kMmaHeads) * p.s.Hk * p.B;
    const size_t smem =
        sizeof(float) * ((p.bias ? (size_t)kMmaHeads * p.s.buckets : 0) + (size_t)kMmaWarps * kMmaHeads * DP);
    attn_decode_mma_kernel<DT, DP><<<(unsigned)grid, kMmaWarps * 32, smem, s>>>(p);
    return cudaGetLastError();
}

template <int DT, int GT>
cudaError_t decode_dim(const AttnDecode& p, cudaStream_t s) {
    constexpr int V = 16 / sizeof(typename Elem<DT>::type);
    const int lanes = (p.s.D + V - 1) / V;
    if (lanes <= 4) return decode<DT, GT, 4, 1>(p, s);
    if (lanes <= 8) return decode<DT, GT, 8, 1>(p, s);
    if (lanes <= 16) return decode<DT, GT, 16, 1>(p, s);
    if constexpr (DT == DT_F32) {
        if (lanes <= 32) return decode<DT, GT, 32, 1>(p, s);
        return decode<DT, GT, 32, 2>(p, s);
    } else {
        return decode<DT, GT, 32, 1>(p, s);
    }
}

template <int DT>
cudaError_t decode_type(const AttnDecode& p, cudaStream_t s) {
    cudaError_t e = cudaErrorInvalidValue;
    bool mma = false;
    if constexpr (DT != DT_F32) {
        mma = p.vec && p.s.D <= 128;
        if (mma) e = p.s.D <= 64 ? decode_mma<DT, 64>(p, s) : decode_mma<DT, 128>(p, s);
    }
    if (!mma) switch (attn_decode_heads(p.s.G)) {
        case 1: e = decode_dim<DT, 1>(p, s); break;
        case 2: e = decode_dim<DT, 2>(p, s); break;
        case 4: e = decode_dim<DT, 4>(p, s); break;
        default: e = decode_dim<DT, 8>(p, s); break;
    }
    if (e != cudaSuccess || p.splits == 1) return e;
    attn_decode_join_kernel<DT><<<(unsigned)(p.B * p.s.H), 128, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

int attn_decode_heads(int G) { return G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : 8; }

cudaError_t launch_attn_append(const AttnAppend& p, cudaStream_t s) {
    const unsigned grid = (unsigned)((p.N + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
    if (p.index64)
        attn_append_kernel<int64_t><<<grid, kAppendThreads, 0, s>>>(p);
    else
        attn_append_kernel<int32_t><<<grid, kAppendThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_attn_decode(const AttnDecode& p, cudaStream_t s) {
    if (p.s.dtype == DT_F32) return decode_type<DT_F32>(p, s);
    if (p.s.dtype == DT_F16) return decode_type<DT_F16>(p, s);
    return decode_type<DT_BF16>(p, s);
}

}  // namespace tbe
