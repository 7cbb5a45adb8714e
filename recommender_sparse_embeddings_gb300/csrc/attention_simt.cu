// Attention over ragged histories, fp32 arithmetic on the FMA units: the
// path of fp32 tensors and of rows the tensor-core kernels do not take.
//
// One CTA takes one tile of T tokens of one history and one head, holds its
// rows in shared memory as fp32 and walks the visible tiles of the other
// side once.  256 threads form a 16 x 16 grid; a thread holds an R x R block
// of logits (R = T / 16; rows ty*R + r, columns tx + 16 c) and an R x D/16
// block of each accumulator, so a step of four products reads 2R 16-byte
// words of shared memory for 4 R^2 FMAs (R = 4: 64): FMA-bound.
// T = 64 up to head_dim 128, 32 above (the tiles must fit 227 KB).
#include <type_traits>

#include "attention.cuh"

namespace tbe {

namespace {

constexpr int kThreads = 256;
static_assert(kMaxBuckets <= kThreads, "a thread per bucket");

template <int T, int DP>
struct Tile {
    static constexpr int LD = DP + 4;  // row stride: the 16 rows a warp reads fall on distinct banks
    static constexpr int PLD = T + 4;
    static constexpr size_t bytes = sizeof(float) * T * LD;
    static constexpr size_t pbytes = sizeof(float) * T * PLD;
};

// Rows of a tile that a history of `len` tokens has, rounded up to 16 (the
// step of a thread's columns); loads, products and sums leave out the rest.
template <int T>
__device__ __forceinline__ int rows_of(int len, int first) {
    return tmin(T, (len - first + 15) / 16 * 16);
}

// Rows [first, first + rows_of) of a history (zeros from `len` on, and beyond
// column D) into a shared tile as fp32.
template <int DT, int T, int DP>
__device__ __forceinline__ void load_tile(float* dst, const Rows& r, int64_t token0, int head, int first, int len,
                                          int D, int vec) {
    using E = typename Elem<DT>::type;
    constexpr int V = 16 / sizeof(E);
    constexpr int LD = Tile<T, DP>::LD;
    const E* base = static_cast<const E*>(r.data) + head * r.head_stride;
    const int rows = rows_of<T>(len, first);
    if (vec) {
        for (int c = threadIdx.x; c < rows * (DP / V); c += kThreads) {
            const int row = c / (DP / V), col = c % (DP / V) * V;
            float f[V];
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = 0.f;
            if (first + row < len && col < D) {
                const E* p = base + (token0 + first + row) * r.token_stride + col;
                unpack16<DT>(__ldg(reinterpret_cast<const uint4*>(p)), f);
            }
#pragma unroll
            for (int i = 0; i < V; i += 4)
                *reinterpret_cast<float4*>(dst + row * LD + col + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
        }
    } else {
        for (int c = threadIdx.x; c < rows * DP; c += kThreads) {
            const int row = c / DP, col = c % DP;
            float f = 0.f;
            if (first + row < len && col < D) f = load_elem<DT>(base, (token0 + first + row) * r.token_stride + col);
            dst[row * LD + col] = f;
        }
    }
}

// acc[r][c] += sum_d a[ty*R + r][d] * b[tx + 16 c][d], for columns below `cols`
template <int T, int DP, bool FULL>
__device__ __forceinline__ void dot_columns(float (&acc)[T / 16][T / 16], const float* a, const float* b, int tx, int ty,
                                         int cols) {
    constexpr int R = T / 16, LD = Tile<T, DP>::LD;
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        float4 x[R], y[R];
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = *reinterpret_cast<const float4*>(a + (ty * R + r) * LD + d);
#pragma unroll
        for (int c = 0; c < R; ++c)
            if (FULL || 16 * c < cols) y[c] = *reinterpret_cast<const float4*>(b + (tx + 16 * c) * LD + d);
#pragma unroll
        for (int c = 0; c < R; ++c)
            if (FULL || 16 * c < cols)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    acc[r][c] = fmaf(x[r].x, y[c].x, acc[r][c]);
                    acc[r][c] = fmaf(x[r].y, y[c].y, acc[r][c]);
                    acc[r][c] = fmaf(x[r].z, y[c].z, acc[r][c]);
                    acc[r][c] = fmaf(x[r].w, y[c].w, acc[r][c]);
                }
    }
}

// (a whole tile without the columns' tests, which cost its inner loop 30 %)
template <int T, int DP>
__device__ __forceinline__ void dot_tile(float (&acc)[T / 16][T / 16], const float* a, const float* b, int tx, int ty,
                                         int cols) {
    if (cols == T)
        dot_columns<T, DP, true>(acc, a, b, tx, ty, T);
    else
        dot_columns<T, DP, false>(acc, a, b, tx, ty, cols);
}

// acc[r][u] (columns 64 u + 4 tx ..) += sum_{j < rows} p[ty*R + r][j] * b[j][column]
template <int T, int DP, bool FULL>
__device__ __forceinline__ void mul_rows(float4 (&acc)[T / 16][DP / 64], const float* p, const float* b, int tx,
                                         int ty, int rows) {
    constexpr int R = T / 16, LD = Tile<T, DP>::LD, PLD = Tile<T, DP>::PLD, U = DP / 64;
#pragma unroll 2
    for (int j = 0; j < (FULL ? T : rows); j += 4) {
        float w[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float4 x = *reinterpret_cast<const float4*>(p + (ty * R + r) * PLD + j);
            w[r][0] = x.x;
            w[r][1] = x.y;
            w[r][2] = x.z;
            w[r][3] = x.w;
        }
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float4 y = *reinterpret_cast<const float4*>(b + (j + jj) * LD + u * 64 + tx * 4);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    acc[r][u].x = fmaf(w[r][jj], y.x, acc[r][u].x);
                    acc[r][u].y = fmaf(w[r][jj], y.y, acc[r][u].y);
                    acc[r][u].z = fmaf(w[r][jj], y.z, acc[r][u].z);
                    acc[r][u].w = fmaf(w[r][jj], y.w, acc[r][u].w);
                }
            }
    }
}

template <int T, int DP>
__device__ __forceinline__ void mul_tile(float4 (&acc)[T / 16][DP / 64], const float* p, const float* b, int tx, int ty,
                                         int rows) {
    if (rows == T)
        mul_rows<T, DP, true>(acc, p, b, tx, ty, T);
    else
        mul_rows<T, DP, false>(acc, p, b, tx, ty, rows);
}

template <int DT, int T, int DP>
__device__ __forceinline__ void store_rows(void* out, const float4 (&acc)[T / 16][DP / 64], const float (&mul)[T / 16],
                                           int64_t token0, int heads, int head, int first, int len, int D, int tx,
                                           int ty) {
    constexpr int R = T / 16, U = DP / 64;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = first + ty * R + r;
        if (row >= len) continue;
        const int64_t at = ((token0 + row) * heads + head) * D;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = u * 64 + tx * 4;
            const float f[4] = {acc[r][u].x, acc[r][u].y, acc[r][u].z, acc[r][u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (col + i < D) store_elem<DT>(out, at + col + i, f[i] * mul[r]);
        }
    }
}

// The key tiles a query tile sees: [0, sink_tiles) and [lo, hi).
template <int T>
__device__ __forceinline__ void key_tiles(const AttnShape& s, int tile, int& sink_tiles, int& lo) {
    const int64_t first = (int64_t)tile * T - s.window + 1;  // first key the tile's first query sees
    lo = first > 0 ? (int)(first / T) : 0;
    sink_tiles = s.sinks > 0 ? tmin((s.sinks + T - 1) / T, lo) : 0;
}

// The bias of every distance the tile pair can have, in base 2:
// bt[x] belongs to distance base + x - (T - 1), x in [0, 2T - 1).
template <int DT, int T>
__device__ __forceinline__ void load_bias(float* bt, const AttnShape& s, const void* bias, int head, int base) {
    for (int x = threadIdx.x; x < 2 * T - 1; x += kThreads) {
        const int d = base + x - (T - 1);
        bt[x] = d >= 0 ? bias_base2(load_elem<DT>(bias, (int64_t)attn_bucket(s, d) * s.H + head)) : 0.f;
    }
}

// Whether the head has a bias of large magnitude; the whole CTA calls it.
template <int DT>
__device__ __forceinline__ bool any_coarse(const AttnShape& s, const void* bias, int head) {
    return __syncthreads_or(threadIdx.x < s.buckets &&
                            attn_coarse(bias_base2(load_elem<DT>(bias, (int64_t)threadIdx.x * s.H + head))));
}

template <int DT, int T, int DP>
__global__ void __launch_bounds__(kThreads) attn_fwd_simt_kernel(const AttnForward p) {
    constexpr int R = T / 16, U = DP / 64, PLD = Tile<T, DP>::PLD;
    extern __shared__ __align__(16) float sm[];
    float* qs = sm;
    float* ks = qs + Tile<T, DP>::bytes / 4;
    float* vs = ks + Tile<T, DP>::bytes / 4;
    float* ps = vs + Tile<T, DP>::bytes / 4;
    float* bt = ps + Tile<T, DP>::pbytes / 4;
    const int64_t w = blockIdx.x / p.s.H;
    const int head = (int)(blockIdx.x % p.s.H);
    AttnItem it;
    if (!find_item(p.src, w, it)) return;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16, kvh = head / p.s.G;
    const int first = it.tile * T;
    const float c2 = p.s.scale * kLog2e;
    const bool coarse = p.bias && any_coarse<DT>(p.s, p.bias, head);
    load_tile<DT, T, DP>(qs, p.q, it.start, head, first, it.len, p.s.D, p.vec);
    float4 o[R][U];
    float m[R], l[R], off[R];  // off: taken off the row's biases
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
        off[r] = 0.f;
        if (coarse) {
            float top = attn_bias_top(p.s, first + ty * R + r, tx, 16, [&](int b) {
                return bias_base2(load_elem<DT>(p.bias, (int64_t)b * p.s.H + head));
            });
#pragma unroll
            for (int o2 = 8; o2 > 0; o2 >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o2, 16));
            off[r] = attn_bias_off(top);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) o[r][u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    int sink_tiles, lo;
    key_tiles<T>(p.s, it.tile, sink_tiles, lo);
    const int steps = sink_tiles + it.tile + 1 - lo;
    const bool active = first + ty / 2 * 2 * R < it.len;  // the warp has a row that exists
    for (int st = 0; st < steps; ++st) {
        const int kt = st < sink_tiles ? st : lo + st - sink_tiles;
        __syncthreads();
        load_tile<DT, T, DP>(ks, p.k, it.start, kvh, kt * T, it.len, p.s.D, p.vec);
        load_tile<DT, T, DP>(vs, p.v, it.start, kvh, kt * T, it.len, p.s.D, p.vec);
        if (p.bias) load_bias<DT, T>(bt, p.s, p.bias, head, (it.tile - kt) * T);
        __syncthreads();
        if (!active) continue;
        const int cols = rows_of<T>(it.len, kt * T);
        float s[R][R];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < R; ++c) s[r][c] = 0.f;
        dot_tile<T, DP>(s, qs, ks, tx, ty, cols);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = first + ty * R + r;
            float top = m[r];
#pragma unroll
            for (int c = 0; c < R; ++c) {
                const int jj = tx + 16 * c, j = kt * T + jj;
                float x = s[r][c] * c2;
                if (p.bias) x += bt[ty * R + r - jj + T - 1] - off[r];
                s[r][c] = attn_visible(i - j, j, p.s.window, p.s.sinks) ? x : -INFINITY;
                top = fmaxf(top, s[r][c]);
            }
#pragma unroll
            for (int o2 = 8; o2 > 0; o2 >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o2, 16));
            const float safe = top == -INFINITY ? 0.f : top;  // no visible key yet
            const float keep = ex2(m[r] - safe);
            m[r] = top;
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < R; ++c) {
                const float e = ex2(s[r][c] - safe);
                sum += e;
                ps[(ty * R + r) * PLD + tx + 16 * c] = e;
            }
#pragma unroll
            for (int o2 = 8; o2 > 0; o2 >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o2, 16);
            l[r] = l[r] * keep + sum;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                o[r][u].x *= keep;
                o[r][u].y *= keep;
                o[r][u].z *= keep;
                o[r][u].w *= keep;
            }
        }
        __syncwarp();  // a warp reads only the rows of ps that it wrote
        mul_tile<T, DP>(o, ps, vs, tx, ty, cols);
    }
    float inv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        inv[r] = l[r] == 0.f ? 0.f : 1.f / l[r];  // a row that sees nothing is zero
        const int row = first + ty * R + r;
        if (tx == 0 && row < it.len) p.lse[(int64_t)head * p.N + it.start + row] = off[r] + (m[r] + log2f(l[r]));
    }
    store_rows<DT, T, DP>(p.out, o, inv, it.start, p.s.H, head, first, it.len, p.s.D, tx, ty);
}

// dq of one query tile, delta of its rows, and the tile's share of the bias
// gradient.  The bias gradient adds ds along diagonals (one distance each) in
// a fixed order: a thread per diagonal of the tile pair, then a thread per
// bucket over the bucket's diagonals, so results do not vary between runs.
template <int DT, int T, int DP>
__global__ void __launch_bounds__(kThreads) attn_dq_simt_kernel(const AttnBackward p) {
    constexpr int R = T / 16, U = DP / 64, PLD = Tile<T, DP>::PLD;
    extern __shared__ __align__(16) float sm[];
    float* qs = sm;
    float* gs = qs + Tile<T, DP>::bytes / 4;
    float* ks = gs + Tile<T, DP>::bytes / 4;
    float* vs = ks + Tile<T, DP>::bytes / 4;
    float* ps = vs + Tile<T, DP>::bytes / 4;
    float* bt = ps + Tile<T, DP>::pbytes / 4;
    float* diag = bt + 2 * T;
    const int64_t w = blockIdx.x / p.s.H;
    const int head = (int)(blockIdx.x % p.s.H);
    AttnItem it;
    if (!find_item(p.src, w, it)) return;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16, kvh = head / p.s.G;
    const int first = it.tile * T;
    const float c2 = p.s.scale * kLog2e;
    load_tile<DT, T, DP>(qs, p.q, it.start, head, first, it.len, p.s.D, p.vec);
    load_tile<DT, T, DP>(gs, p.g, it.start, head, first, it.len, p.s.D, p.vec);
    const Rows orows{p.out, (int64_t)p.s.H * p.s.D, p.s.D};
    load_tile<DT, T, DP>(ks, orows, it.start, head, first, it.len, p.s.D, p.vec);
    __syncthreads();
    float4 acc[R][U];
    float lse[R], delta[R], excess[R];
    bool large = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = ty * R + r;
        float t = 0.f;
        for (int d = tx; d < DP; d += 16) t = fmaf(gs[row * Tile<T, DP>::LD + d], ks[row * Tile<T, DP>::LD + d], t);
#pragma unroll
        for (int o2 = 8; o2 > 0; o2 >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o2, 16);
        delta[r] = t;
        excess[r] = 0.f;
        lse[r] = INFINITY;
        if (first + row < it.len) {
            const int64_t at = (int64_t)head * p.N + it.start + first + row;
            const float x = p.lse[at];
            lse[r] = attn_no_weights(x) ? INFINITY : x;  // then all its weights are 2^-inf
            large |= attn_coarse(x);
            if (tx == 0) p.delta[at] = t;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) acc[r][u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mine = 0.f;  // bias gradient of bucket threadIdx.x
    int sink_tiles, lo;
    key_tiles<T>(p.s, it.tile, sink_tiles, lo);
    const int steps = sink_tiles + it.tile + 1 - lo;
    // 16-bit out: g . out misses delta by out's rounding, so a first sweep
    // adds up sum_j p (dp - g . out) in fp32, which is what it misses.  The
    // same sweep adds up the weights of rows whose |lse| is large.
    const bool active = first + ty / 2 * 2 * R < it.len;  // the warp has a row that exists
    constexpr bool kTwice = DT != DT_F32;
    const bool twice = __syncthreads_or(large) || kTwice;
    float over[R] = {}, z[R] = {};
    for (int st = twice ? -steps : 0; st < steps; ++st) {
        if (st == 0 && twice) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int o2 = 8; o2 > 0; o2 >>= 1) {
                    over[r] += __shfl_xor_sync(0xffffffffu, over[r], o2, 16);
                    z[r] += __shfl_xor_sync(0xffffffffu, z[r], o2, 16);
                }
                const bool of_row = attn_coarse(lse[r]);
                if (of_row) {
                    over[r] /= z[r];
                    excess[r] = log2f(z[r]);
                }
                if (kTwice || of_row) delta[r] += over[r];
                const int row = first + ty * R + r;
                if (tx == 0 && row < it.len) {
                    const int64_t at = (int64_t)head * p.N + it.start + row;
                    p.delta[at] = delta[r];
                    if (of_row) p.excess[at] = excess[r];
                }
            }
        }
        const int tile = st < 0 ? st + steps : st;
        const int kt = tile < sink_tiles ? tile : lo + tile - sink_tiles;
        const int base = (it.tile - kt) * T;
        __syncthreads();
        load_tile<DT, T, DP>(ks, p.k, it.start, kvh, kt * T, it.len, p.s.D, p.vec);
        load_tile<DT, T, DP>(vs, p.v, it.start, kvh, kt * T, it.len, p.s.D, p.vec);
        if (p.bias) load_bias<DT, T>(bt, p.s, p.bias, head, base);
        __syncthreads();
        float s[R][R], dp[R][R];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < R; ++c) s[r][c] = dp[r][c] = 0.f;
        const int cols = rows_of<T>(it.len, kt * T);
        if (active) {
            dot_tile<T, DP>(s, qs, ks, tx, ty, cols);
            dot_tile<T, DP>(dp, gs, vs, tx, ty, cols);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = first + ty * R + r;
#pragma unroll
            for (int c = 0; c < R; ++c) {
                const int jj = tx + 16 * c, j = kt * T + jj;
                const float b = p.bias ? bt[ty * R + r - jj + T - 1] : 0.f;
                const float x = s[r][c] * c2 + ((b - lse[r]) - excess[r]);
                const bool seen = i < it.len && attn_visible(i - j, j, p.s.window, p.s.sinks);
                const float e = seen ? ex2(x) : 0.f;
                const float ds = seen && !attn_lone(i, j, p.s.window, p.s.sinks) ? e * (dp[r][c] - delta[r]) : 0.f;
                if (st < 0) {
                    over[r] += ds;
                    z[r] += e;
                }
                ps[(ty * R + r) * PLD + jj] = ds;
            }
        }
        if (st < 0) continue;
        __syncthreads();
        if (active) mul_tile<T, DP>(acc, ps, ks, tx, ty, cols);
        if (p.bias) {
            for (int x = threadIdx.x; x < 2 * T - 1; x += kThreads) {
                const int off = x - (T - 1);  // row - column
                float t = 0.f;
                for (int j = tmax(0, -off); j < tmin(T, T - off); ++j) t += ps[(j + off) * PLD + j];
                diag[x] = t;
            }
            __syncthreads();
            if (threadIdx.x < p.s.buckets) {
                const int from = tmax(__ldg(p.s.starts + threadIdx.x), tmax(0, base - (T - 1)));
                const int to = tmin(__ldg(p.s.starts + threadIdx.x + 1), base + T);
                for (int d = from; d < to; ++d) mine += diag[d - base + T - 1];
            }
        }
    }
    float mul[R];
#pragma unroll
    for (int r = 0; r < R; ++r) mul[r] = p.s.scale;
    store_rows<DT, T, DP>(p.gq, acc, mul, it.start, p.s.H, head, first, it.len, p.s.D, tx, ty);
    if (p.bias && threadIdx.x < p.s.buckets) p.bias_part[(w * p.s.H + head) * p.s.buckets + threadIdx.x] = mine;
}

// dk and dv of one key tile and key-value head: the sums over the group's
// query heads and the visible query tiles, in a fixed order.  Here the
// logits' rows are keys and their columns queries.
template <int DT, int T, int DP>
__global__ void __launch_bounds__(kThreads) attn_dkv_simt_kernel(const AttnBackward p) {
    constexpr int R = T / 16, U = DP / 64, PLD = Tile<T, DP>::PLD;
    extern __shared__ __align__(16) float sm[];
    float* ks = sm;
    float* vs = ks + Tile<T, DP>::bytes / 4;
    float* qs = vs + Tile<T, DP>::bytes / 4;
    float* gs = qs + Tile<T, DP>::bytes / 4;
    float* ps = gs + Tile<T, DP>::bytes / 4;
    float* bt = ps + Tile<T, DP>::pbytes / 4;
    float* ls = bt + 2 * T;
    float* de = ls + T;
    float* ex = de + T;
    const int64_t w = blockIdx.x / p.s.Hk;
    const int kvh = (int)(blockIdx.x % p.s.Hk);
    AttnItem it;
    if (!find_item(p.src, w, it)) return;
    const int kt = it.tiles - 1 - it.tile;  // the first tiles are seen most: they start first
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int first = kt * T;
    const float c2 = p.s.scale * kLog2e;
    load_tile<DT, T, DP>(ks, p.k, it.start, kvh, first, it.len, p.s.D, p.vec);
    load_tile<DT, T, DP>(vs, p.v, it.start, kvh, first, it.len, p.s.D, p.vec);
    float4 dk[R][U], dv[R][U];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int u = 0; u < U; ++u) dk[r][u] = dv[r][u] = make_float4(0.f, 0.f, 0.f, 0.f);
    // last query that sees a key of the tile: window - 1 tokens after its last key, or the last of all for sinks
    const int64_t last = first < p.s.sinks ? it.len - 1 : tmin<int64_t>(it.len - 1, (int64_t)first + T - 1 + p.s.window - 1);
    const int qt_end = (int)(last / T) + 1;
    const bool active = first + ty / 2 * 2 * R < it.len;  // the warp has a row that exists
    for (int g = 0; g < p.s.G; ++g) {
        const int head = kvh * p.s.G + g;
        for (int qt = kt; qt < qt_end; ++qt) {
            __syncthreads();
            load_tile<DT, T, DP>(qs, p.q, it.start, head, qt * T, it.len, p.s.D, p.vec);
            load_tile<DT, T, DP>(gs, p.g, it.start, head, qt * T, it.len, p.s.D, p.vec);
            if (p.bias) load_bias<DT, T>(bt, p.s, p.bias, head, (qt - kt) * T);
            if (threadIdx.x < T) {
                const int i = qt * T + threadIdx.x;
                float x = INFINITY, y = 0.f, z = 0.f;
                if (i < it.len) {
                    const int64_t at = (int64_t)head * p.N + it.start + i;
                    x = p.lse[at];
                    y = p.delta[at];
                    if (attn_coarse(x)) z = p.excess[at];
                    if (attn_no_weights(x)) x = INFINITY;
                }
                ls[threadIdx.x] = x;
                de[threadIdx.x] = y;
                ex[threadIdx.x] = z;
            }
            __syncthreads();
            if (!active) continue;
            const int cols = rows_of<T>(it.len, qt * T);
            float s[R][R], dp[R][R];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < R; ++c) s[r][c] = dp[r][c] = 0.f;
            dot_tile<T, DP>(s, ks, qs, tx, ty, cols);
            dot_tile<T, DP>(dp, vs, gs, tx, ty, cols);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int j = first + ty * R + r;
#pragma unroll
                for (int c = 0; c < R; ++c) {
                    const int ii = tx + 16 * c, i = qt * T + ii;
                    const float b = p.bias ? bt[ii - (ty * R + r) + T - 1] : 0.f;
                    const float x = s[r][c] * c2 + ((b - ls[ii]) - ex[ii]);
                    const bool seen = i < it.len && attn_visible(i - j, j, p.s.window, p.s.sinks);
                    const float e = seen ? ex2(x) : 0.f;
                    ps[(ty * R + r) * PLD + ii] = e;
                    const bool live = seen && !attn_lone(i, j, p.s.window, p.s.sinks);
                    s[r][c] = live ? e * (dp[r][c] - de[ii]) : 0.f;
                }
            }
            __syncwarp();  // a warp reads only the rows of ps that it wrote
            mul_tile<T, DP>(dv, ps, gs, tx, ty, cols);
            __syncwarp();
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < R; ++c) ps[(ty * R + r) * PLD + tx + 16 * c] = s[r][c];
            __syncwarp();
            mul_tile<T, DP>(dk, ps, qs, tx, ty, cols);
        }
    }
    float one[R], mul[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        one[r] = 1.f;
        mul[r] = p.s.scale;
    }
    store_rows<DT, T, DP>(p.gv, dv, one, it.start, p.s.Hk, kvh, first, it.len, p.s.D, tx, ty);
    store_rows<DT, T, DP>(p.gk, dk, mul, it.start, p.s.Hk, kvh, first, it.len, p.s.D, tx, ty);
}

// Exclusive sum over the CTA's 1024 threads, and the total (64 bits: offsets
// that overlap can name far more tiles than N tokens have).
__device__ __forceinline__ int64_t block_scan(int64_t n, int64_t* warp_sum, int64_t& all) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int64_t before = 0;
    all = 0;
    for (int k = 0; k < 32; ++k) {
        if (k < warp) before += warp_sum[k];
        all += warp_sum[k];
    }
    __syncthreads();
    return before + incl - n;
}

// Work items of the batch, and the offsets' check: histories of n tiles of
// `tile` tokens, each history's last tile first.  One CTA; 1024 histories a
// pass.  A history whose offsets are not ordered within [0, N] gets no item.
template <typename I>
__global__ void __launch_bounds__(1024) attn_items_kernel(const I* __restrict__ off, int64_t N, int B, int tile,
                                                          AttnItem* __restrict__ items, int64_t capacity,
                                                          int32_t* n_items, uint32_t* error, const FarWork far) {
    __shared__ int64_t warp_sum[32];
    __shared__ int32_t far_count;  // far items written: the first ones, all of them where the offsets are in order
    if (threadIdx.x == 0) far_count = 0;
    const int lane = threadIdx.x % 32;
    int64_t base = 0, far_base = 0, slot_base = 0;
    for (int b0 = 0; b0 < B; b0 += 1024) {
        const int b = b0 + threadIdx.x;
        int64_t lo = 0, hi = 0;
        if (b < B) {
            lo = (int64_t)off[b];
            hi = (int64_t)off[b + 1];
            const bool bad = lo < 0 || hi < lo || hi > N;
            if (bad || (b == 0 && lo != 0) || (b == B - 1 && hi != N)) atomicOr(error, ERR_OFFSETS);
            if (bad) hi = lo = 0;
        }
        int64_t all;
        const int n = (int)((hi - lo + tile - 1) / tile);
        const int64_t at = base + block_scan(n, warp_sum, all);
        base += all;
        int slot = -1;
        if (far.most > 0) {
            // chunks of the query blocks behind the first tile's window, where there are many
            const int behind = (int)((hi - lo + 63) / 64) - far.near;
            const int chunks = behind > far.blocks ? (behind + far.blocks - 1) / far.blocks : 0;
            const int64_t here = far_base + block_scan(chunks, warp_sum, all);
            far_base += all;
            const int64_t first = slot_base + block_scan(chunks > 0 ? chunks + 1 : 0, warp_sum, all);
            slot_base += all;
            if (chunks > 0 && here + chunks <= far.most) {
                slot = (int)first;
                atomicMax(&far_count, (int32_t)here + chunks);
                for (int c = 0; c < chunks; ++c)
                    far.items[here + c] = FarItem{(int)lo, (int)(hi - lo), c, chunks, slot, {0, 0, 0}};
            }
        }
        // short histories' items by their own lanes, a long one's by the warp
        constexpr int kOwn = 8;
        const int own = n <= kOwn ? n : 0;
        for (int t = 0; t < own; ++t)
            if (at + t < capacity) {
                items[at + t] = AttnItem{(int)lo, (int)(hi - lo), n - 1 - t, n};
                if (far.most > 0) far.slot_of[at + t] = slot;
            }
        for (uint32_t left = __ballot_sync(0xffffffffu, n > kOwn); left; left &= left - 1) {
            const int k = __ffs(left) - 1;
            const int nk = __shfl_sync(0xffffffffu, n, k);
            const int64_t ak = __shfl_sync(0xffffffffu, at, k);
            const int sk = (int)__shfl_sync(0xffffffffu, lo, k);
            const int lk = (int)(__shfl_sync(0xffffffffu, hi, k)) - sk;
            const int pk = __shfl_sync(0xffffffffu, slot, k);
            for (int t = lane; t < nk; t += 32)
                if (ak + t < capacity) {
                    items[ak + t] = AttnItem{sk, lk, nk - 1 - t, nk};
                    if (far.most > 0) far.slot_of[ak + t] = pk;
                }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        *n_items = (int32_t)tmin<int64_t>(base, capacity);
        if (far.most > 0) *far.n_items = far_count;
    }
}

// grad_bias[bucket, head] = the items' shares added up in a fixed order: a
// warp per (bucket, head), its lanes over the items, then a tree.
template <int DT>
__global__ void __launch_bounds__(256) attn_bias_reduce_kernel(const float* __restrict__ part,
                                                               const ItemSource src, int64_t max_items,
                                                               const int32_t* __restrict__ n_far, int H,
                                                               int buckets, void* grad_bias) {
    const int pair = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (pair >= H * buckets) return;
    const int head = pair / buckets, b = pair % buckets;
    // (offsets that overlap can name more tiles than there is room for)
    const int n = (int)tmin<int64_t>(count_items(src), max_items);
    float t = 0.f;
    for (int w = lane; w < n; w += 32) t += part[((int64_t)w * H + head) * buckets + b];
    const int nf = n_far ? *n_far : 0;
    for (int w = lane; w < nf; w += 32) t += part[((max_items + w) * H + head) * buckets + b];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) store_elem<DT>(grad_bias, (int64_t)b * H + head, t);
}

template <int T, int DP>
constexpr size_t fwd_smem() {
    return 3 * Tile<T, DP>::bytes + Tile<T, DP>::pbytes + sizeof(float) * 2 * T;
}
template <int T, int DP>
constexpr size_t bwd_smem() {
    return 4 * Tile<T, DP>::bytes + Tile<T, DP>::pbytes + sizeof(float) * 5 * T;
}

template <typename K>
cudaError_t allow(K kernel, size_t bytes, int optin) {
    if (bytes > (size_t)optin) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int DT, int T, int DP>
cudaError_t configure(int optin) {
    cudaError_t e = allow(attn_fwd_simt_kernel<DT, T, DP>, fwd_smem<T, DP>(), optin);
    if (e == cudaSuccess) e = allow(attn_dq_simt_kernel<DT, T, DP>, bwd_smem<T, DP>(), optin);
    if (e == cudaSuccess) e = allow(attn_dkv_simt_kernel<DT, T, DP>, bwd_smem<T, DP>(), optin);
    return e;
}

template <int DT, int T, int DP>
cudaError_t forward(const AttnForward& p, int64_t n, cudaStream_t s) {
    attn_fwd_simt_kernel<DT, T, DP><<<(unsigned)(n * p.s.H), kThreads, fwd_smem<T, DP>(), s>>>(p);
    return cudaGetLastError();
}

template <int DT, int T, int DP>
cudaError_t backward(const AttnBackward& p, int64_t n, cudaStream_t s) {
    attn_dq_simt_kernel<DT, T, DP><<<(unsigned)(n * p.s.H), kThreads, bwd_smem<T, DP>(), s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    attn_dkv_simt_kernel<DT, T, DP><<<(unsigned)(n * p.s.Hk), kThreads, bwd_smem<T, DP>(), s>>>(p);
    return cudaGetLastError();
}

}  // namespace

// Tokens a tile.  64 up to head_dim 128, 32 above (the tiles must fit shared
// memory).  fp32 batches that would leave SMs without a CTA take 32 as well:
// more and shorter CTAs (40 fp32 histories of 93 tokens, 2 heads: forward and
// backward 185 us with 64, 152 with 32; 64 histories of 190, 4 heads, which
// fill the SMs: forward 101 us with 64, 108 with 32).
int attn_simt_tile(int dtype, int D, int H, int64_t N, int64_t B, int num_sms) {
    if (D > 128) return 32;
    return dtype == DT_F32 && ((N / 64 + B) * H < 2 * (int64_t)num_sms || N < 32 * B) ? 32 : 64;
}

cudaError_t attn_simt_configure(int optin) {
    cudaError_t e = cudaSuccess;
    auto all = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (e == cudaSuccess) e = configure<DT, 64, 64>(optin);
        if (e == cudaSuccess) e = configure<DT, 64, 128>(optin);
        if (e == cudaSuccess) e = configure<DT, 32, 256>(optin);
        if constexpr (DT == DT_F32) {
            if (e == cudaSuccess) e = configure<DT, 32, 64>(optin);
            if (e == cudaSuccess) e = configure<DT, 32, 128>(optin);
        }
    };
    all(std::integral_constant<int, DT_F32>{});
    all(std::integral_constant<int, DT_F16>{});
    all(std::integral_constant<int, DT_BF16>{});
    return e;
}

#define ATTN_BY_TYPE_AND_DIM(CALL)                                          \
    do {                                                                    \
        const int D = p.s.D, tile = p.src.tile;                             \
        if (p.s.dtype == DT_F32) {                                          \
            if (D <= 64 && tile == 32) return CALL<DT_F32, 32, 64>(p, max_items, s);   \
            if (D <= 128 && tile == 32) return CALL<DT_F32, 32, 128>(p, max_items, s); \
            if (D <= 64) return CALL<DT_F32, 64, 64>(p, max_items, s);      \
            if (D <= 128) return CALL<DT_F32, 64, 128>(p, max_items, s);    \
            return CALL<DT_F32, 32, 256>(p, max_items, s);                  \
        } else if (p.s.dtype == DT_F16) {                                   \
            if (D <= 64) return CALL<DT_F16, 64, 64>(p, max_items, s);      \
            if (D <= 128) return CALL<DT_F16, 64, 128>(p, max_items, s);    \
            return CALL<DT_F16, 32, 256>(p, max_items, s);                  \
        } else {                                                            \
            if (D <= 64) return CALL<DT_BF16, 64, 64>(p, max_items, s);     \
            if (D <= 128) return CALL<DT_BF16, 64, 128>(p, max_items, s);   \
            return CALL<DT_BF16, 32, 256>(p, max_items, s);                 \
        }                                                                   \
    } while (0)

cudaError_t launch_attn_forward_simt(const AttnForward& p, int64_t max_items, cudaStream_t s) {
    ATTN_BY_TYPE_AND_DIM(forward);
}

cudaError_t launch_attn_backward_simt(const AttnBackward& p, int64_t max_items, cudaStream_t s) {
    ATTN_BY_TYPE_AND_DIM(backward);
}

cudaError_t launch_attn_items(const void* offsets, int index64, int64_t N, int B, int tile, AttnItem* items,
                              int64_t capacity, int32_t* n_items, uint32_t* error, const FarWork& far,
                              cudaStream_t s) {
    if (index64)
        attn_items_kernel<int64_t><<<1, 1024, 0, s>>>(static_cast<const int64_t*>(offsets), N, B, tile, items, capacity,
                                                      n_items, error, far);
    else
        attn_items_kernel<int32_t><<<1, 1024, 0, s>>>(static_cast<const int32_t*>(offsets), N, B, tile, items, capacity,
                                                      n_items, error, far);
    return cudaGetLastError();
}

cudaError_t launch_attn_bias_reduce(const AttnBackward& p, void* grad_bias, cudaStream_t s) {
    const int grid = (p.s.H * p.s.buckets + 7) / 8;
    const int32_t* far = p.far.most > 0 ? p.far.n_items : nullptr;
    if (p.s.dtype == DT_F32)
        attn_bias_reduce_kernel<DT_F32><<<grid, 256, 0, s>>>(p.bias_part, p.src, p.max_items, far, p.s.H, p.s.buckets,
                                                               grad_bias);
    else if (p.s.dtype == DT_F16)
        attn_bias_reduce_kernel<DT_F16><<<grid, 256, 0, s>>>(p.bias_part, p.src, p.max_items, far, p.s.H, p.s.buckets,
                                                               grad_bias);
    else
        attn_bias_reduce_kernel<DT_BF16><<<grid, 256, 0, s>>>(p.bias_part, p.src, p.max_items, far, p.s.H, p.s.buckets,
                                                               grad_bias);
    return cudaGetLastError();
}

}  // namespace tbe
