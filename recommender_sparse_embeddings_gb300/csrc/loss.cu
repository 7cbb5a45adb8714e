// Softmax cross entropy of rows over a table of items, and its gradients.
// Declarations, formulas and contracts are in include/tbe.h.
#include <algorithm>
#include <new>

#include <nvtx3/nvToolsExt.h>

#include "../../include/tbe.h"
#include "tbe_internal.cuh"

namespace tbe {
int cuda_fail(cudaError_t e);
}

using namespace tbe;

struct tbe_softmax_loss {
    int device = 0;
    int num_sms = 0;
    tbe_softmax_loss_config c{};
    uint32_t* error = nullptr;
};

namespace {

constexpr int kMaxLossDim = 4096;
constexpr int kChunk = 4096;  // items of a piece of the backward pass

struct CallRange {
    explicit CallRange(const char* name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange&) = delete;
    CallRange& operator=(const CallRange&) = delete;
};

struct Loss {
    const void *x, *table, *targets;
    int64_t x_stride, table_stride, N, V;
    int index64, D;
    float scale;
    float *loss, *lse;  // forward: written; backward: lse is read
    const float* g;
    void *gx, *gw;
    float *d, *sum;  // [N][kChunk], [N][D]
    int64_t v0, v1;  // the piece
    uint32_t* error;
};

// The row's item; -1 for a row that is left out.
__device__ __forceinline__ int64_t target_of(const Loss& p, int64_t i) {
    const int64_t t = p.index64 ? static_cast<const int64_t*>(p.targets)[i] : static_cast<const int32_t*>(p.targets)[i];
    if (t >= p.V) {
        atomicOr(p.error, ERR_OOB);
        return -1;
    }
    return t < 0 ? -1 : t;
}

// acc[a][b] = sum_k A(m0 + 4 ty + a, k) B(k, n0 + 4 tx + b) of a 64 x 64 tile.
template <typename FA, typename FB>
__device__ __forceinline__ void tile_product(float (&acc)[4][4], int64_t K, FA A, FB B) {
    __shared__ float sa[16][65], sb[16][65];
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = 0.f;
    for (int64_t k0 = 0; k0 < K; k0 += 16) {
        __syncthreads();
        for (int x = threadIdx.x; x < 1024; x += 256) {
            sa[x % 16][x / 16] = k0 + x % 16 < K ? A(x / 16, k0 + x % 16) : 0.f;
            sb[x % 16][x / 16] = k0 + x % 16 < K ? B(k0 + x % 16, x / 16) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(sa[k][4 * ty + a], sb[k][4 * tx + b], acc[a][b]);
    }
}

template <int DT>
__device__ __forceinline__ void tile_scores(const Loss& p, float (&s)[4][4], int64_t m0, int64_t n0) {
    tile_product(
        s, p.D,
        [&](int m, int64_t k) { return m0 + m < p.N ? load_elem<DT>(p.x, (m0 + m) * p.x_stride + k) : 0.f; },
        [&](int64_t k, int n) { return n0 + n < p.V ? load_elem<DT>(p.table, (n0 + n) * p.table_stride + k) : 0.f; });
}

template <int DT>
__global__ void __launch_bounds__(256) loss_forward_kernel(const Loss p) {
    const int64_t m0 = (int64_t)blockIdx.x * 64;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float m[4];
    double l[4];  // (fp32 would lose 2^-24 of the sum per item)
    for (int a = 0; a < 4; ++a) m[a] = -INFINITY, l[a] = 0.;
    for (int64_t n0 = 0; n0 < p.V; n0 += 64) {
        float s[4][4];
        tile_scores<DT>(p, s, m0, n0);
        for (int a = 0; a < 4; ++a)
            for (int b = 0; b < 4; ++b)
                if (n0 + 4 * tx + b < p.V) {
                    const float y = s[a][b] * p.scale, to = fmaxf(m[a], y);
                    l[a] = l[a] * expf(m[a] - to) + expf(y - to);
                    m[a] = to;
                }
    }
    for (int a = 0; a < 4; ++a) {
        for (int o = 8; o > 0; o /= 2) {
            const float mo = __shfl_xor_sync(0xffffffffu, m[a], o), to = fmaxf(m[a], mo);
            const double lo = __shfl_xor_sync(0xffffffffu, l[a], o);
            l[a] = (l[a] == 0. ? 0. : l[a] * expf(m[a] - to)) + (lo == 0. ? 0. : lo * expf(mo - to));
            m[a] = to;
        }
        const int64_t i = m0 + 4 * ty + a;
        if (tx == 0 && i < p.N) {
            p.lse[i] = m[a] + logf((float)l[a]);
            const int64_t t = target_of(p, i);
            float y = 0.f;
            if (t >= 0)
                for (int k = 0; k < p.D; ++k)
                    y = fmaf(load_elem<DT>(p.x, i * p.x_stride + k), load_elem<DT>(p.table, t * p.table_stride + k), y);
            p.loss[i] = t < 0 ? 0.f : (m[a] - y * p.scale) + logf((float)l[a]);
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(256) loss_d_kernel(const Loss p) {
    const int64_t m0 = (int64_t)blockIdx.x * 64, n0 = p.v0 + (int64_t)blockIdx.y * 64;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float s[4][4];
    tile_scores<DT>(p, s, m0, n0);
    for (int a = 0; a < 4; ++a) {
        const int64_t i = m0 + 4 * ty + a;
        if (i >= p.N) continue;
        const int64_t t = target_of(p, i);
        for (int b = 0; b < 4; ++b) {
            const int64_t v = n0 + 4 * tx + b;
            if (v < p.v1)
                p.d[i * kChunk + v - p.v0] =
                    t < 0 ? 0.f : p.g[i] * p.scale * (expf(s[a][b] * p.scale - p.lse[i]) - (v == t ? 1.f : 0.f));
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(256) loss_gx_kernel(const Loss p) {
    const int64_t m0 = (int64_t)blockIdx.x * 64, n0 = (int64_t)blockIdx.y * 64;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float s[4][4];
    tile_product(
        s, p.v1 - p.v0, [&](int m, int64_t k) { return m0 + m < p.N ? p.d[(m0 + m) * kChunk + k] : 0.f; },
        [&](int64_t k, int n) {
            return n0 + n < p.D ? load_elem<DT>(p.table, (p.v0 + k) * p.table_stride + n0 + n) : 0.f;
        });
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const int64_t i = m0 + 4 * ty + a, j = n0 + 4 * tx + b;
            if (i >= p.N || j >= p.D) continue;
            const float y = (p.v0 > 0 ? p.sum[i * p.D + j] : 0.f) + s[a][b];
            p.sum[i * p.D + j] = y;
            if (p.v1 == p.V) store_elem<DT>(p.gx, i * p.D + j, y);
        }
}

template <int DT>
__global__ void __launch_bounds__(256) loss_gw_kernel(const Loss p) {
    const int64_t m0 = (int64_t)blockIdx.x * 64, n0 = (int64_t)blockIdx.y * 64;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float s[4][4];
    tile_product(
        s, p.N, [&](int m, int64_t k) { return p.v0 + m0 + m < p.v1 ? p.d[k * kChunk + m0 + m] : 0.f; },
        [&](int64_t k, int n) {
            return n0 + n < p.D && target_of(p, k) >= 0 ? load_elem<DT>(p.x, k * p.x_stride + n0 + n) : 0.f;
        });
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const int64_t v = p.v0 + m0 + 4 * ty + a, j = n0 + 4 * tx + b;
            if (v < p.v1 && j < p.D) store_elem<DT>(p.gw, v * p.D + j, s[a][b]);
        }
}

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }
bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }
int status(cudaError_t e) { return e == cudaSuccess ? TBE_OK : cuda_fail(e); }

bool on_device(const tbe_softmax_loss* h) {
    int d = -1;
    return cudaGetDevice(&d) == cudaSuccess && d == h->device;
}

bool within_limits(int64_t N, int64_t V) { return N < (int64_t(1) << 30) && V <= (int64_t(1) << 31) - 1024; }

int check(const tbe_softmax_loss* h, const void* x, int64_t x_stride, const void* table, int64_t table_stride,
          const void* targets, int32_t index_dtype, int64_t N, int64_t V) {
    if (!h || !on_device(h)) return TBE_ERR_INVALID_ARG;
    if (index_dtype != TBE_I32 && index_dtype != TBE_I64) return TBE_ERR_INVALID_ARG;
    if (N < 0 || V < 0 || (N > 0 && (V == 0 || !x || !table || !targets))) return TBE_ERR_INVALID_ARG;
    if (x_stride < 0 || (V > 1 && table_stride < h->c.dim)) return TBE_ERR_INVALID_ARG;
    return within_limits(N, V) ? TBE_OK : TBE_ERR_UNSUPPORTED;
}

template <int DT>
cudaError_t launch_backward(Loss p, cudaStream_t s) {
    const unsigned mt = (unsigned)((p.N + 63) / 64), dt = (unsigned)((p.D + 63) / 64);
    for (p.v0 = 0; p.v0 < p.V; p.v0 = p.v1) {
        p.v1 = std::min<int64_t>(p.V, p.v0 + kChunk);
        const unsigned vt = (unsigned)((p.v1 - p.v0 + 63) / 64);
        loss_d_kernel<DT><<<dim3(mt, vt), 256, 0, s>>>(p);
        if (p.gx) loss_gx_kernel<DT><<<dim3(mt, dt), 256, 0, s>>>(p);
        if (p.gw) loss_gw_kernel<DT><<<dim3(vt, dt), 256, 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace

extern "C" {

int tbe_softmax_loss_create(const tbe_softmax_loss_config* c, tbe_softmax_loss** out) {
    CallRange range("tbe_softmax_loss_create");
    if (!out) return TBE_ERR_INVALID_ARG;
    *out = nullptr;
    if (!c) return TBE_ERR_INVALID_ARG;
    if (c->dtype != TBE_F32 && c->dtype != TBE_F16 && c->dtype != TBE_BF16) return TBE_ERR_INVALID_ARG;
    if (c->dim <= 0 || !(c->scale > 0.f && c->scale - c->scale == 0.f)) return TBE_ERR_INVALID_ARG;
    if (c->dim > kMaxLossDim) return TBE_ERR_UNSUPPORTED;
    tbe_softmax_loss* h = new (std::nothrow) tbe_softmax_loss();
    if (!h) return TBE_ERR_NO_MEMORY;
    h->c = *c;
    cudaError_t e = cudaGetDevice(&h->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
    if (e == cudaSuccess) e = cudaMalloc(&h->error, 16);
    if (e == cudaSuccess) e = cudaMemset(h->error, 0, 16);
    if (e != cudaSuccess) {
        if (h->error) cudaFree(h->error);
        delete h;
        return e == cudaErrorMemoryAllocation ? TBE_ERR_NO_MEMORY : cuda_fail(e);
    }
    *out = h;
    return TBE_OK;
}

void tbe_softmax_loss_destroy(tbe_softmax_loss* h) {
    if (!h) return;
    if (h->error) cudaFree(h->error);
    delete h;
}

size_t tbe_softmax_loss_workspace_bytes(const tbe_softmax_loss* h, int64_t N, int64_t V, int32_t backward) {
    if (!h || N < 0 || V < 0 || !within_limits(N, V)) return 0;
    return 256 + (backward ? align_up(sizeof(float) * N * kChunk) + align_up(sizeof(float) * N * h->c.dim) : 0);
}

int tbe_softmax_loss_forward(tbe_softmax_loss* h, const void* x, int64_t x_stride, const void* table,
                             int64_t table_stride, const void* targets, int32_t index_dtype, int64_t N, int64_t V,
                             float* loss, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range("tbe_softmax_loss_forward");
    const int rc = check(h, x, x_stride, table, table_stride, targets, index_dtype, N, V);
    if (rc) return rc;
    if (!workspace || !aligned16(workspace) || (N > 0 && (!loss || !lse))) return TBE_ERR_INVALID_ARG;
    if (workspace_bytes < tbe_softmax_loss_workspace_bytes(h, N, V, 0)) return TBE_ERR_WORKSPACE_TOO_SMALL;
    if (N == 0) return TBE_OK;
    Loss p{};
    p.x = x, p.table = table, p.targets = targets, p.x_stride = x_stride, p.table_stride = table_stride;
    p.N = N, p.V = V, p.index64 = index_dtype == TBE_I64, p.D = h->c.dim, p.scale = h->c.scale;
    p.loss = loss, p.lse = lse, p.error = h->error;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)((N + 63) / 64);
    if (h->c.dtype == TBE_F32)
        loss_forward_kernel<DT_F32><<<grid, 256, 0, s>>>(p);
    else if (h->c.dtype == TBE_F16)
        loss_forward_kernel<DT_F16><<<grid, 256, 0, s>>>(p);
    else
        loss_forward_kernel<DT_BF16><<<grid, 256, 0, s>>>(p);
    return status(cudaGetLastError());
}

int tbe_softmax_loss_backward(tbe_softmax_loss* h, const void* x, int64_t x_stride, const void* table,
                              int64_t table_stride, const void* targets, int32_t index_dtype, int64_t N, int64_t V,
                              const float* lse, const float* grad_loss, void* grad_x, void* grad_table,
                              void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range("tbe_softmax_loss_backward");
    const int rc = check(h, x, x_stride, table, table_stride, targets, index_dtype, N, V);
    if (rc) return rc;
    if (!workspace || !aligned16(workspace) || (N > 0 && (!lse || !grad_loss))) return TBE_ERR_INVALID_ARG;
    if (workspace_bytes < tbe_softmax_loss_workspace_bytes(h, N, V, 1)) return TBE_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) {
        if (!grad_table || V == 0) return TBE_OK;
        return status(cudaMemsetAsync(grad_table, 0, (size_t)V * h->c.dim * elem_bytes(h->c.dtype), s));
    }
    Loss p{};
    p.x = x, p.table = table, p.targets = targets, p.x_stride = x_stride, p.table_stride = table_stride;
    p.N = N, p.V = V, p.index64 = index_dtype == TBE_I64, p.D = h->c.dim, p.scale = h->c.scale;
    p.lse = const_cast<float*>(lse), p.g = grad_loss, p.gx = grad_x, p.gw = grad_table, p.error = h->error;
    char* at = reinterpret_cast<char*>(align_up(reinterpret_cast<uintptr_t>(workspace)));
    p.d = reinterpret_cast<float*>(at);
    p.sum = reinterpret_cast<float*>(at + align_up(sizeof(float) * N * kChunk));
    return status(h->c.dtype == TBE_F32   ? launch_backward<DT_F32>(p, s)
                  : h->c.dtype == TBE_F16 ? launch_backward<DT_F16>(p, s)
                                          : launch_backward<DT_BF16>(p, s));
}

int tbe_softmax_loss_get_error(tbe_softmax_loss* h, void* stream) {
    if (!h || !on_device(h)) return TBE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t bits = 0;
    cudaError_t e = cudaMemcpyAsync(&bits, h->error, sizeof bits, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = cudaMemsetAsync(h->error, 0, sizeof bits, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e);
    if (bits & ERR_TIMEOUT) return TBE_ERR_TIMEOUT;
    if (bits & ERR_OOB) return TBE_ERR_INDEX_OOB;
    return TBE_OK;
}

}  // extern "C"
