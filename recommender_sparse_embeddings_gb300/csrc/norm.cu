// Layer norm of rows, with the residual sum taken on the way, and its
// gradients.  Declarations, formulas and contracts are in include/tbe.h.
#include <algorithm>
#include <cfloat>
#include <new>

#include <nvtx3/nvToolsExt.h>

#include "../../include/tbe.h"
#include "tbe_internal.cuh"

namespace tbe {
int cuda_fail(cudaError_t e);
}

using namespace tbe;

struct tbe_layer_norm {
    int device = 0;
    int num_sms = 0;
    tbe_layer_norm_config c{};
};

namespace {

constexpr int kMaxNormDim = 16384;
// CTAs of the backward kernel per SM at most: bounds its partial sums.  Wide rows'
// CTAs are large: two fit (8192 x 4096 f16 with one 73 us, with two 60); of narrow
// rows 4, 8 and 16 take the same time.
constexpr int most_ctas(int D) { return D <= 512 ? 8 : 2; }

struct CallRange {
    explicit CallRange(const char* name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange&) = delete;
    CallRange& operator=(const CallRange&) = delete;
};

struct NormForward {
    const void *x, *residual, *weight, *bias;
    int64_t x_stride, residual_stride, rows;
    int D;
    float eps;
    void *out, *total;
    float* stats;
};

struct NormBackward {
    const void *total, *g, *u, *weight;
    int64_t total_stride, g_stride, u_stride, rows;
    const float* stats;
    int D;
    void *gx, *gw, *gb;
    float* part;  // [CTAs][2][D]: sums of g xhat and of g over a CTA's rows
};

// Both kernels stream rows that stay in registers from the first sum to the
// store: T threads hold a row, thread t the accesses t, t + T, ... (K of them) of E
// consecutive elements (16 bytes, or one element where rows are not aligned).
// A group of T <= 32 lanes sums by shuffles alone, a larger one through shared
// memory and a barrier of its own.  Groups take rows in turn (the grid fills the GPU
// once), so weights stay in registers and the next rows are fetched before this
// one's sums.
template <int DT, int E>
struct Access {
    using Raw = uint4;
};
template <>
struct Access<DT_F32, 1> {
    using Raw = float;
};
template <>
struct Access<DT_F16, 1> {
    using Raw = unsigned short;
};
template <>
struct Access<DT_BF16, 1> {
    using Raw = unsigned short;
};

template <int DT, int E>
using Raw = typename Access<DT, E>::Raw;

template <int DT, int E>
__device__ __forceinline__ void to_floats(const Raw<DT, E>& r, float* f) {
    if constexpr (E > 1)
        unpack16<DT>(r, f);
    else if constexpr (DT == DT_F32)
        f[0] = r;
    else
        f[0] = DT == DT_F16 ? h_bits_to_float(r) : bf16_bits_to_float(r);
}

template <int DT>
__device__ __forceinline__ uint32_t pair_bits(float a, float b) {
    uint32_t r;
    if constexpr (DT == DT_F16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

template <int DT, int E>
__device__ __forceinline__ Raw<DT, E> from_floats(const float* f) {
    if constexpr (DT == DT_F32) {
        if constexpr (E == 1)
            return f[0];
        else
            return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                              __float_as_uint(f[3]));
    } else if constexpr (E == 1) {
        return (unsigned short)pair_bits<DT>(f[0], 0.f);
    } else {
        return make_uint4(pair_bits<DT>(f[0], f[1]), pair_bits<DT>(f[2], f[3]), pair_bits<DT>(f[4], f[5]),
                          pair_bits<DT>(f[6], f[7]));
    }
}

// The thread's K accesses of one row of D elements, zeros behind its end.
template <int DT, int E, int K, int T>
struct RowPart {
    Raw<DT, E> r[K];

    __device__ __forceinline__ void load(const void* base, int64_t at, int D, int t) {
        const Raw<DT, E>* p =
            reinterpret_cast<const Raw<DT, E>*>(static_cast<const char*>(base) + at * elem_bytes(DT));
#pragma unroll
        for (int k = 0; k < K; ++k) {
            r[k] = Raw<DT, E>{};
            if ((k * T + t) * E < D) r[k] = __ldg(p + k * T + t);
        }
    }
    __device__ __forceinline__ void store(void* base, int64_t at, int D, int t) const {
        Raw<DT, E>* p = reinterpret_cast<Raw<DT, E>*>(static_cast<char*>(base) + at * elem_bytes(DT));
#pragma unroll
        for (int k = 0; k < K; ++k)
            if ((k * T + t) * E < D) p[k * T + t] = r[k];
    }
    __device__ __forceinline__ void get(float* f) const {
#pragma unroll
        for (int k = 0; k < K; ++k) to_floats<DT, E>(r[k], f + k * E);
    }
    __device__ __forceinline__ void set(const float* f) {
#pragma unroll
        for (int k = 0; k < K; ++k) r[k] = from_floats<DT, E>(f + k * E);
    }
};

// Threads of a CTA: several groups where a row leaves room for them (they share
// the backward pass's partial sums of the weights; the forward pass wants the
// registers).
constexpr int forward_threads(int T) { return T <= 32 ? 256 : T; }
constexpr int backward_threads(int T) { return T <= 32 ? 256 : T == 128 ? 512 : T; }

// The backward pass's rows that a group takes in turn, fetched ahead.  16-byte
// accesses go through shared memory, S rows deep: a thread copies its own accesses
// there (cp.async) and reads them back, so nothing has to wait for another
// thread, and rows in flight take no registers (50,523 x 512 bf16 54 -> 44 us; the
// forward pass has registers for the next row and lost 5 % by it).  Single elements
// and rows of a CTA each are held in registers, one row ahead (8192 x 4096 f16 58
// us, through shared memory 62).
template <int DT, int E, int K, int T>
struct Feed {
    using Part = RowPart<DT, E, K, T>;
    static constexpr int kThreads = backward_threads(T), kAccess = kThreads * 16;
    static constexpr bool kRing = E > 1 && T < 256;
    static constexpr int S = K == 1 ? 5 : K == 2 ? 4 : 2;
    static constexpr size_t kBytes = kRing ? (size_t)S * 3 * K * kAccess : 0;
    const NormBackward& p;
    const int64_t step;
    const int t;
    int at;
    uint32_t room;  // of this thread
    Part x, g, u;   // without the ring: the next row

    __device__ __forceinline__ Feed(const NormBackward& args, int64_t step, int t)
        : p(args), step(step), t(t), at(0), room(0) {}

    __device__ __forceinline__ void copy_one(const void* base, int64_t at, uint32_t to) {
        const char* from = static_cast<const char*>(base) + at * elem_bytes(DT);
#pragma unroll
        for (int k = 0; k < K; ++k)  // (behind the row's end: nothing read, zeros)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + k * kAccess),
                         "l"((k * T + t) * E < p.D ? from + (k * T + t) * 16 : from), "r"((k * T + t) * E < p.D ? 16 : 0)
                         : "memory");
    }

    __device__ __forceinline__ void copy(int64_t row, int slot) {
        if (row < p.rows) {
            const uint32_t to = room + slot * (3 * K * kAccess);
            copy_one(p.total, row * p.total_stride, to);
            copy_one(p.g, row * p.g_stride, to + K * kAccess);
            if (p.u) copy_one(p.u, row * p.u_stride, to + 2 * K * kAccess);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    __device__ __forceinline__ void load(int64_t row) {
        if (row >= p.rows) {  // a group without a row adds nothing to the sums
            x = g = Part{};
            return;
        }
        x.load(p.total, row * p.total_stride, p.D, t);
        g.load(p.g, row * p.g_stride, p.D, t);
        if (p.u) u.load(p.u, row * p.u_stride, p.D, t);
    }

    __device__ __forceinline__ void start(unsigned char* smem, int64_t row) {
        if constexpr (kRing) {
            room = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + threadIdx.x * 16;
#pragma unroll
            for (int i = 0; i < S - 1; ++i) copy(row + i * step, i);
        } else {
            load(row);
        }
    }

    // The ring's row `row` is there.
    __device__ __forceinline__ void take(int64_t row) {
        copy(row + (S - 1) * step, (at + S - 1) % S);
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    }
    __device__ __forceinline__ void get(int i, float* f) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            uint4 v;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(room + ((at * 3 + i) * K + k) * kAccess)
                         : "memory");
            unpack16<DT>(v, f + k * E);
        }
    }
    __device__ __forceinline__ void leave() { at = (at + 1) % S; }
};

// Sums of N values over the T threads of a row, in all of them.  Wider groups
// than a warp join through shared memory; `turn` alternates between its two
// halves, so one barrier a sum is enough.
template <int T, int kGroups, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int& turn) {
#pragma unroll
    for (int o = (T < 32 ? T : 32) / 2; o > 0; o /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (T > 32) {
        __shared__ float part[2][kGroups][N][T / 32];
        const int group = threadIdx.x / T;
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) part[turn][group][i][threadIdx.x % T / 32] = v[i];
        if constexpr (kGroups > 1)
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(T) : "memory");
        else
            __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = part[turn][group][i][threadIdx.x % (T / 32)];
#pragma unroll
            for (int o = T / 64; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
            v[i] = s;
        }
        turn ^= 1;
    }
}

template <int DT, int E, int K, int T>
__global__ void __launch_bounds__(forward_threads(T)) norm_forward_kernel(const NormForward p) {
    using Part = RowPart<DT, E, K, T>;
    constexpr int kGroups = forward_threads(T) / T, M = E * K;
    const int t = threadIdx.x % T;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    const float width = p.D, per = 1.f / width;
    Part w{}, b{};
    if (p.weight) w.load(p.weight, 0, p.D, t);
    if (p.bias) b.load(p.bias, 0, p.D, t);
    int64_t row = (int64_t)blockIdx.x * kGroups + threadIdx.x / T;
    Part x{}, r{};
    auto fetch = [&](int64_t i) {
        if (i >= p.rows) return;
        x.load(p.x, i * p.x_stride, p.D, t);
        if (p.residual) r.load(p.residual, i * p.residual_stride, p.D, t);
    };
    fetch(row);
    int turn = 0;
    // (the groups of a warp run alike: its first row decides)
    for (; row - threadIdx.x % 32 / T < p.rows; row += step) {
        float f[M], s[1] = {0.f};
        x.get(f);
        Part keep{};
        if (p.residual) {
            float q[M];
            r.get(q);
#pragma unroll
            for (int i = 0; i < M; ++i) f[i] += q[i];
            keep.set(f);
            keep.get(f);
        }
        fetch(row + step);
#pragma unroll
        for (int i = 0; i < M; ++i) s[0] += f[i];
        row_sums<T, kGroups>(s, turn);
        const float about = s[0] * per;
        const float mean = fmaf(fmaf(-width, about, s[0]), per, about);  // (the sum / D, rounded once)
        s[0] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if ((k * T + t) * E < p.D)
#pragma unroll
                for (int i = k * E; i < k * E + E; ++i) {
                    f[i] -= mean;
                    s[0] = fmaf(f[i], f[i], s[0]);
                }
        row_sums<T, kGroups>(s, turn);
        const float rstd = rsqrtf(fmaf(s[0], per, p.eps));
        if (row >= p.rows) continue;
        if (p.residual) keep.store(p.total, row * p.D, p.D, t);
        float q[M];
#pragma unroll
        for (int i = 0; i < M; ++i) f[i] *= rstd;
        if (p.weight) {
            w.get(q);
#pragma unroll
            for (int i = 0; i < M; ++i) f[i] *= q[i];
        }
        if (p.bias) {
            b.get(q);
#pragma unroll
            for (int i = 0; i < M; ++i) f[i] += q[i];
        }
        keep.set(f);
        keep.store(p.out, row * p.D, p.D, t);
        if (t == 0) {
            p.stats[row] = mean;
            p.stats[p.rows + row] = rstd;
        }
    }
}

// Wide rows of 1024 threads keep the weights' sums in shared memory: they have at
// most 64 registers a thread, and those of more than 8 elements spill as it is (164 to
// 268 bytes with 16-bit accesses of 16 bytes, 0.4 to 1.6 KB with fp32's or single
// elements, as do other variants of single elements above 512 columns by 0.1 to 0.4).
template <int T>
constexpr bool sums_in_smem() {
    return T == 1024;
}

template <int DT, int E, int K, int T>
__global__ void __launch_bounds__(backward_threads(T)) norm_backward_kernel(const NormBackward p) {
    using Part = RowPart<DT, E, K, T>;
    constexpr int kThreads = backward_threads(T), kGroups = kThreads / T, M = E * K;
    constexpr bool kSmem = sums_in_smem<T>();
    using Rows = Feed<DT, E, K, T>;
    extern __shared__ __align__(16) unsigned char smem[];
    // behind the rows ahead (kSmem: [2 M][threads]) or, after them, in their place (several groups: [M][threads])
    float* room = reinterpret_cast<float*>(smem + (kSmem ? Rows::kBytes : 0));
    const int t = threadIdx.x % T;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    const float per = 1.f / p.D;
    const bool params = p.gw || p.gb;
    Part w{};
    if (p.weight) w.load(p.weight, 0, p.D, t);
    int64_t row = (int64_t)blockIdx.x * kGroups + threadIdx.x / T;
    Rows feed(p, step, t);
    feed.start(smem, row);
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](int64_t i) {
        mean = i < p.rows ? __ldg(p.stats + i) : 0.f;
        rstd = i < p.rows ? __ldg(p.stats + p.rows + i) : 0.f;
    };
    float sw[kSmem ? 1 : M], sb[kSmem ? 1 : M];
    if constexpr (kSmem) {
#pragma unroll
        for (int i = 0; i < 2 * M; ++i) room[i * kThreads + threadIdx.x] = 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < M; ++i) sw[i] = sb[i] = 0.f;
    }
    fetch(row);
    int turn = 0;
    for (; row - threadIdx.x % 32 / T < p.rows; row += step) {
        float h[M], a[M], q[M], s[2] = {0.f, 0.f};
        const float m = mean, is = rstd;
        const bool valid = row < p.rows;
        Part on{};
        if constexpr (Rows::kRing) {
            feed.take(row);
            feed.get(0, h);
            feed.get(1, a);
            if (T < 32 && !valid)
#pragma unroll
                for (int i = 0; i < M; ++i) a[i] = h[i] = 0.f;
        } else {
            feed.x.get(h);
            feed.g.get(a);
            on = feed.u;
            feed.load(row + step);
        }
        fetch(row + step);
        // Accesses behind the row's end hold g = 0, and their xhat -m * is meets nothing
        // else; but it has to be finite.  It is, unless all elements are m exactly (one
        // that is not is an fp32 step away: is <= sqrt(D) 2^24 / m), and then any number
        // serves their xhat, 0.  (A mask in the loop cost rows of 256 threads 10 to 25 %.)
        const float to_hat = fabsf(m * is) <= FLT_MAX ? is : 0.f;
#pragma unroll
        for (int i = 0; i < M; ++i) {
            h[i] = (h[i] - m) * to_hat;
            if constexpr (kSmem) {
                if (params) {
                    room[i * kThreads + threadIdx.x] = fmaf(a[i], h[i], room[i * kThreads + threadIdx.x]);
                    room[(M + i) * kThreads + threadIdx.x] += a[i];
                }
            } else {
                sw[i] = fmaf(a[i], h[i], sw[i]);
                sb[i] += a[i];
            }
        }
        if (p.weight) {
            w.get(q);
#pragma unroll
            for (int i = 0; i < M; ++i) a[i] *= q[i];
        }
#pragma unroll
        for (int i = 0; i < M; ++i) {
            s[0] += a[i];
            s[1] = fmaf(a[i], h[i], s[1]);
        }
        row_sums<T, kGroups>(s, turn);
        s[0] *= per;
        s[1] *= per;
        if (p.u) {
            if constexpr (Rows::kRing)
                feed.get(2, q);
            else
                on.get(q);
#pragma unroll
            for (int i = 0; i < M; ++i) a[i] = fmaf(is, (a[i] - s[0]) - h[i] * s[1], q[i]);
        } else {
#pragma unroll
            for (int i = 0; i < M; ++i) a[i] = is * ((a[i] - s[0]) - h[i] * s[1]);
        }
        if constexpr (Rows::kRing) feed.leave();
        on.set(a);
        if (valid) on.store(p.gx, row * p.D, p.D, t);
    }
    if constexpr (Rows::kRing) asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!params) return;
    // the CTA's sums of both kinds, its groups in order
    float* part = p.part + (int64_t)blockIdx.x * 2 * p.D;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
        if constexpr (kGroups > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < M; ++i) room[i * kThreads + threadIdx.x] = kind ? sb[i] : sw[i];
            __syncthreads();
        }
        // element k * T * E + t * E + e of the row: sum i = k * E + e of thread t
        for (int y = threadIdx.x; y < M * T; y += kThreads) {
            const int i = y / T, lane = y % T, j = (i / E) * T * E + lane * E + i % E;
            if (j >= p.D) continue;
            float v = 0.f;
            if constexpr (kGroups > 1) {
#pragma unroll
                for (int o = 0; o < kGroups; ++o) v += room[i * kThreads + o * T + lane];
            } else if constexpr (kSmem) {
                v = room[(kind * M + i) * kThreads + lane];
            } else {
#pragma unroll
                for (int z = 0; z < M; ++z)
                    if (z == i) v = kind ? sb[z] : sw[z];
            }
            part[(int64_t)kind * p.D + j] = v;
        }
    }
}

// The CTAs' partial sums joined: 32 columns a CTA, 32 of its threads share a
// column's partials and add up their sums in order.
template <int DT>
__global__ void __launch_bounds__(1024) norm_join_kernel(const NormBackward p, int parts) {
    chain_wait();
    __shared__ float s[32][33];
    const int j = blockIdx.x * 32 + threadIdx.x % 32, lane = threadIdx.x / 32;
    float v = 0.f;
    if (j < 2 * p.D)
#pragma unroll 4
        for (int i = lane; i < parts; i += 32) v += p.part[(int64_t)i * 2 * p.D + j];
    s[lane][threadIdx.x % 32] = v;
    __syncthreads();
    v = s[threadIdx.x % 32][lane];
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int column = blockIdx.x * 32 + lane;
    if (threadIdx.x % 32 != 0 || column >= 2 * p.D) return;
    void* to = column < p.D ? p.gw : p.gb;
    if (to) store_elem<DT>(to, column < p.D ? column : column - p.D, v);
}

bool on_device(const tbe_layer_norm* h) {
    int d = -1;
    return cudaGetDevice(&d) == cudaSuccess && d == h->device;
}

// Whether a block shares bytes with one of `rows` rows of `row` bytes, `stride` apart.
bool over_rows(const void* block, int64_t bytes, const void* base, int64_t stride, int64_t row, int64_t rows) {
    if (!block || !base || (uintptr_t)base >= (uintptr_t)block + (uintptr_t)bytes) return false;
    const int64_t behind = (int64_t)((uintptr_t)block - (uintptr_t)base) - row;  // its start from the first row's end
    if (behind < 0) return true;
    const int64_t first = stride > 0 ? behind / stride + 1 : rows;  // the first row that ends behind its start
    return first < rows && (uintptr_t)base + (uintptr_t)(first * stride) < (uintptr_t)block + (uintptr_t)bytes;
}

// Whether a result of contiguous rows may not lie where it does beside an operand:
// over the same rows it may (a row is read before it is written, by the same
// threads), over others of them it may not.
bool misplaced(const tbe_layer_norm* h, const void* result, const void* operand, int64_t stride, int64_t rows) {
    const int64_t e = elem_bytes(h->c.dtype), row = h->c.dim * e;
    if (result == operand && (stride == h->c.dim || rows == 1)) return false;
    return over_rows(result, rows * row, operand, stride * e, row, rows);
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

bool vec_rows(const tbe_layer_norm* h, const void* p, int64_t stride) {
    const int e = elem_bytes(h->c.dtype);
    return aligned16(p) && stride * e % 16 == 0 && h->c.dim * e % 16 == 0;
}

// CTAs that fill the GPU once, no more than the rows need.
unsigned fill(const tbe_layer_norm* h, int per_sm, int groups, int64_t rows) {
    return (unsigned)std::min<int64_t>((rows + groups - 1) / groups, (int64_t)per_sm * h->num_sms);
}

template <typename F>
int resident(F kernel, int threads, size_t smem) {
    int ctas = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, kernel, threads, smem) != cudaSuccess) return 1;
    return std::max(ctas, 1);
}

template <int DT, int E, int K, int T>
cudaError_t forward(const NormForward& p, const tbe_layer_norm* h, cudaStream_t s) {
    constexpr int threads = forward_threads(T);
    auto* kernel = norm_forward_kernel<DT, E, K, T>;
    static const int per_sm = resident(kernel, threads, 0);
    kernel<<<fill(h, per_sm, threads / T, p.rows), threads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int DT, int E, int K, int T>
cudaError_t backward(const NormBackward& p, const tbe_layer_norm* h, cudaStream_t s) {
    constexpr int threads = backward_threads(T), M = E * K;
    constexpr size_t ahead = Feed<DT, E, K, T>::kBytes, sums = sizeof(float) * threads * M;
    constexpr size_t smem = sums_in_smem<T>() ? ahead + 2 * sums : threads > T ? std::max(ahead, sums) : ahead;
    auto* kernel = norm_backward_kernel<DT, E, K, T>;
    if (smem > 48 * 1024) {  // (an attribute of the device's copy of the kernel, so set at every call)
        const cudaError_t f = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (f != cudaSuccess) return f;
    }
    static const int per_sm = resident(kernel, threads, smem);
    const unsigned grid = fill(h, std::min(per_sm, most_ctas(p.D)), threads / T, p.rows);
    if (grid > 0) kernel<<<grid, threads, smem, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !(p.gw || p.gb)) return e;
    return launch_chained(norm_join_kernel<DT>, dim3((2 * p.D + 31) / 32), dim3(1024), s, p, (int)grid);
}

// The fewest threads a row whose registers hold it: at most 32 elements a thread
// of 16-bit rows in the forward pass (16 of 1025 to 2048 columns), 16 of fp32 and of
// rows off 16 bytes, and 16 in the backward pass, whose sums take two registers an
// element besides.  fp32's backward pass of 4097 to 8192 columns has 8 (4000 x 8192
// 119 -> 101 us; 16-bit rows lost by it: 8000 x 5000 bf16 110 -> 127, x 8192 131 -> 138).
template <int DT>
cudaError_t launch_forward(const NormForward& p, bool vec, const tbe_layer_norm* h, cudaStream_t s) {
    constexpr int E = DT == DT_F32 ? 4 : 8;
    if (!vec) {
        if (p.D <= 128) return forward<DT, 1, 4, 32>(p, h, s);
        if (p.D <= 512) return forward<DT, 1, 16, 32>(p, h, s);
        if (p.D <= 2048) return forward<DT, 1, 16, 128>(p, h, s);
        if (p.D <= 8192) return forward<DT, 1, 16, 512>(p, h, s);
        return forward<DT, 1, 16, 1024>(p, h, s);
    }
    if (p.D <= 8 * E) return forward<DT, E, 1, 8>(p, h, s);
    if (p.D <= 16 * E) return forward<DT, E, 1, 16>(p, h, s);
    if (p.D <= 32 * E) return forward<DT, E, 1, 32>(p, h, s);
    if (p.D <= 64 * E) return forward<DT, E, 2, 32>(p, h, s);
    if (p.D <= 128 * E) return forward<DT, E, 4, 32>(p, h, s);
    if (p.D <= 256 * E) return forward<DT, E, 2, 128>(p, h, s);
    if (p.D <= 512 * E) return forward<DT, E, 4, 128>(p, h, s);
    if (p.D <= 1024 * E) return forward<DT, E, 4, 256>(p, h, s);
    if (p.D <= 2048 * E) return forward<DT, E, 4, 512>(p, h, s);
    if constexpr (DT == DT_F32) return forward<DT, E, 4, 1024>(p, h, s);
    return cudaErrorInvalidValue;
}

template <int DT>
cudaError_t launch_backward(const NormBackward& p, bool vec, const tbe_layer_norm* h, cudaStream_t s) {
    constexpr int E = DT == DT_F32 ? 4 : 8, K2 = 16 / E;
    if (!vec) {
        if (p.D <= 128) return backward<DT, 1, 4, 32>(p, h, s);
        if (p.D <= 512) return backward<DT, 1, 16, 32>(p, h, s);
        if (p.D <= 2048) return backward<DT, 1, 16, 128>(p, h, s);
        if (p.D <= 8192) return backward<DT, 1, 16, 512>(p, h, s);
        return backward<DT, 1, 16, 1024>(p, h, s);
    }
    if (p.D <= 8 * E) return backward<DT, E, 1, 8>(p, h, s);
    if (p.D <= 16 * E) return backward<DT, E, 1, 16>(p, h, s);
    if (p.D <= 32 * E) return backward<DT, E, 1, 32>(p, h, s);
    if (p.D <= 64 * E) return backward<DT, E, 2, 32>(p, h, s);
    if constexpr (DT == DT_F32) {
        if (p.D <= 512) return backward<DT, E, K2, 32>(p, h, s);
    } else {
        if (p.D <= 1024) return backward<DT, E, 1, 128>(p, h, s);
    }
    if (p.D <= 2048) return backward<DT, E, K2, 128>(p, h, s);
    if (p.D <= 4096) return backward<DT, E, K2, 256>(p, h, s);
    if constexpr (DT == DT_F32) {
        if (p.D <= 8192) return backward<DT, E, K2 / 2, 1024>(p, h, s);
    } else {
        if (p.D <= 8192) return backward<DT, E, K2, 512>(p, h, s);
    }
    return backward<DT, E, K2, 1024>(p, h, s);
}

}  // namespace

extern "C" {

int tbe_layer_norm_create(const tbe_layer_norm_config* c, tbe_layer_norm** out) {
    CallRange range("tbe_layer_norm_create");
    if (!out) return TBE_ERR_INVALID_ARG;
    *out = nullptr;
    if (!c) return TBE_ERR_INVALID_ARG;
    if (c->dtype != TBE_F32 && c->dtype != TBE_F16 && c->dtype != TBE_BF16) return TBE_ERR_INVALID_ARG;
    if (c->dim <= 0 || !(c->eps >= 0.f && c->eps - c->eps == 0.f) || (c->has_weight & ~1) || (c->has_bias & ~1))
        return TBE_ERR_INVALID_ARG;
    if (c->dim > kMaxNormDim) return TBE_ERR_UNSUPPORTED;
    tbe_layer_norm* h = new (std::nothrow) tbe_layer_norm();
    if (!h) return TBE_ERR_NO_MEMORY;
    h->c = *c;
    cudaError_t e = cudaGetDevice(&h->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
    if (e != cudaSuccess) {
        delete h;
        return cuda_fail(e);
    }
    *out = h;
    return TBE_OK;
}

void tbe_layer_norm_destroy(tbe_layer_norm* h) { delete h; }

size_t tbe_layer_norm_workspace_bytes(const tbe_layer_norm* h, int64_t rows) {
    if (!h || rows < 0 || rows >= (int64_t(1) << 31)) return 0;
    const int64_t ctas = std::min<int64_t>(rows, (int64_t)most_ctas(h->c.dim) * h->num_sms);
    return 256 + sizeof(float) * 2 * (size_t)ctas * h->c.dim;
}

int tbe_layer_norm_forward(tbe_layer_norm* h, const void* x, int64_t x_stride, const void* residual,
                           int64_t residual_stride, const void* weight, const void* bias, int64_t rows, void* out,
                           void* total, float* stats, void* stream) {
    CallRange range("tbe_layer_norm_forward");
    if (!h || !on_device(h) || rows < 0 || x_stride < 0 || residual_stride < 0) return TBE_ERR_INVALID_ARG;
    if ((weight != nullptr) != (h->c.has_weight != 0) || (bias != nullptr) != (h->c.has_bias != 0))
        return TBE_ERR_INVALID_ARG;
    if (rows >= (int64_t(1) << 31)) return TBE_ERR_UNSUPPORTED;
    if (rows == 0) return TBE_OK;
    if (!x || !out || !stats || (residual != nullptr) != (total != nullptr)) return TBE_ERR_INVALID_ARG;
    const int64_t e_bytes = elem_bytes(h->c.dtype), row = h->c.dim * e_bytes, stats_bytes = 2 * rows * (int64_t)sizeof(float);
    if (overlap(out, rows * row, total, rows * row) || over_rows(stats, stats_bytes, x, x_stride * e_bytes, row, rows) ||
        over_rows(stats, stats_bytes, residual, residual_stride * e_bytes, row, rows))
        return TBE_ERR_INVALID_ARG;
    for (const void* result : {static_cast<const void*>(out), static_cast<const void*>(total)})
        if (misplaced(h, result, x, x_stride, rows) || misplaced(h, result, residual, residual_stride, rows) ||
            overlap(result, rows * row, weight, row) || overlap(result, rows * row, bias, row) ||
            overlap(result, rows * row, stats, stats_bytes))
            return TBE_ERR_INVALID_ARG;
    if (overlap(stats, stats_bytes, weight, row) || overlap(stats, stats_bytes, bias, row)) return TBE_ERR_INVALID_ARG;
    const NormForward p{x, residual, weight, bias, x_stride, residual_stride, rows, h->c.dim, h->c.eps, out, total, stats};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = vec_rows(h, x, x_stride) && vec_rows(h, out, 0) && (!weight || aligned16(weight)) &&
                     (!bias || aligned16(bias)) &&
                     (!residual || (vec_rows(h, residual, residual_stride) && vec_rows(h, total, 0)));
    const cudaError_t e = h->c.dtype == TBE_F32   ? launch_forward<DT_F32>(p, vec, h, s)
                          : h->c.dtype == TBE_F16 ? launch_forward<DT_F16>(p, vec, h, s)
                                                  : launch_forward<DT_BF16>(p, vec, h, s);
    return e == cudaSuccess ? TBE_OK : cuda_fail(e);
}

int tbe_layer_norm_backward(tbe_layer_norm* h, const void* total, int64_t total_stride, const float* stats,
                            const void* grad_out, int64_t grad_out_stride, const void* grad_total,
                            int64_t grad_total_stride, const void* weight, int64_t rows, void* grad_x,
                            void* grad_weight, void* grad_bias, void* workspace, size_t workspace_bytes,
                            void* stream) {
    CallRange range("tbe_layer_norm_backward");
    if (!h || !on_device(h) || rows < 0 || total_stride < 0 || grad_out_stride < 0 || grad_total_stride < 0)
        return TBE_ERR_INVALID_ARG;
    if ((weight != nullptr) != (h->c.has_weight != 0) || (grad_weight != nullptr) != (h->c.has_weight != 0) ||
        (grad_bias != nullptr) != (h->c.has_bias != 0))
        return TBE_ERR_INVALID_ARG;
    if (rows >= (int64_t(1) << 31)) return TBE_ERR_UNSUPPORTED;
    if (!workspace || !aligned16(workspace)) return TBE_ERR_INVALID_ARG;
    if (rows > 0 && (!total || !stats || !grad_out || !grad_x)) return TBE_ERR_INVALID_ARG;
    if (workspace_bytes < tbe_layer_norm_workspace_bytes(h, rows)) return TBE_ERR_WORKSPACE_TOO_SMALL;
    // (grad_weight and grad_bias are written after all operands are read)
    const int64_t row = h->c.dim * elem_bytes(h->c.dtype);
    if (misplaced(h, grad_x, total, total_stride, rows) || misplaced(h, grad_x, grad_out, grad_out_stride, rows) ||
        misplaced(h, grad_x, grad_total, grad_total_stride, rows) || overlap(grad_x, rows * row, weight, row) ||
        overlap(grad_x, rows * row, stats, 2 * rows * (int64_t)sizeof(float)) || overlap(grad_weight, row, grad_bias, row) ||
        overlap(grad_x, rows * row, grad_weight, row) || overlap(grad_x, rows * row, grad_bias, row))
        return TBE_ERR_INVALID_ARG;
    const NormBackward p{total, grad_out, grad_total, weight, total_stride, grad_out_stride, grad_total_stride, rows,
                         stats, h->c.dim, grad_x, grad_weight, grad_bias, static_cast<float*>(workspace)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = vec_rows(h, total, total_stride) && vec_rows(h, grad_out, grad_out_stride) &&
                     (!grad_total || vec_rows(h, grad_total, grad_total_stride)) && vec_rows(h, grad_x, 0) &&
                     (!weight || aligned16(weight));
    const cudaError_t e = h->c.dtype == TBE_F32   ? launch_backward<DT_F32>(p, vec, h, s)
                          : h->c.dtype == TBE_F16 ? launch_backward<DT_F16>(p, vec, h, s)
                                                  : launch_backward<DT_BF16>(p, vec, h, s);
    return e == cudaSuccess ? TBE_OK : cuda_fail(e);
}

}  // extern "C"
