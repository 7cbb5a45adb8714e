// Layer norm of rows, with the residual sum taken on the way, and its
// gradients.  Declarations, formulas and contracts are in include/tbe.h.
#include <algorithm>
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
constexpr int kThreads = 256;

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
    float* part;  // [CTAs][2][D]
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float cta_sum(float v) {
    __shared__ float part[kThreads / 32];
    v = warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += part[w];
    return t;
}

// One CTA a row, three passes over it.
template <int DT>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const NormForward p) {
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int64_t at = row * p.D;
        const void* t = p.residual ? p.total : p.x;
        const int64_t t0 = p.residual ? at : row * p.x_stride;
        if (p.residual)
            for (int j = threadIdx.x; j < p.D; j += kThreads)
                store_elem<DT>(p.total, at + j,
                               load_elem<DT>(p.x, row * p.x_stride + j) +
                                   load_elem<DT>(p.residual, row * p.residual_stride + j));
        auto value = [&](int j) {  // (written above: no read-only load)
            if constexpr (DT == DT_F32) return static_cast<const float*>(t)[t0 + j];
            if constexpr (DT == DT_F16) return __half2float(static_cast<const __half*>(t)[t0 + j]);
            return __bfloat162float(static_cast<const __nv_bfloat16*>(t)[t0 + j]);
        };
        float s = 0.f;
        for (int j = threadIdx.x; j < p.D; j += kThreads) s += value(j);
        const float mean = cta_sum(s) / p.D;
        s = 0.f;
        for (int j = threadIdx.x; j < p.D; j += kThreads) s += (value(j) - mean) * (value(j) - mean);
        const float rstd = 1.f / sqrtf(cta_sum(s) / p.D + p.eps);
        for (int j = threadIdx.x; j < p.D; j += kThreads)
            store_elem<DT>(p.out, at + j, (value(j) - mean) * rstd * (p.weight ? load_elem<DT>(p.weight, j) : 1.f) +
                                              (p.bias ? load_elem<DT>(p.bias, j) : 0.f));
        if (threadIdx.x == 0) {
            p.stats[row] = mean;
            p.stats[p.rows + row] = rstd;
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(const NormBackward p) {
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const float mean = p.stats[row], rstd = p.stats[p.rows + row];
        float s = 0.f, sx = 0.f;
        for (int j = threadIdx.x; j < p.D; j += kThreads) {
            const float a = load_elem<DT>(p.g, row * p.g_stride + j) * (p.weight ? load_elem<DT>(p.weight, j) : 1.f);
            s += a;
            sx += a * (load_elem<DT>(p.total, row * p.total_stride + j) - mean) * rstd;
        }
        s = cta_sum(s) / p.D;
        sx = cta_sum(sx) / p.D;
        for (int j = threadIdx.x; j < p.D; j += kThreads) {
            const float a = load_elem<DT>(p.g, row * p.g_stride + j) * (p.weight ? load_elem<DT>(p.weight, j) : 1.f);
            const float hat = (load_elem<DT>(p.total, row * p.total_stride + j) - mean) * rstd;
            store_elem<DT>(p.gx, row * p.D + j,
                           rstd * (a - s - hat * sx) + (p.u ? load_elem<DT>(p.u, row * p.u_stride + j) : 0.f));
        }
    }
}

// One thread a column.
template <int DT>
__global__ void __launch_bounds__(kThreads) norm_weight_kernel(const NormBackward p) {
    const int j = blockIdx.x * kThreads + threadIdx.x;
    if (j >= p.D) return;
    float w = 0.f, b = 0.f;
    for (int64_t row = 0; row < p.rows; ++row) {
        const float g = load_elem<DT>(p.g, row * p.g_stride + j);
        w += g * (load_elem<DT>(p.total, row * p.total_stride + j) - p.stats[row]) * p.stats[p.rows + row];
        b += g;
    }
    if (p.gw) store_elem<DT>(p.gw, j, w);
    if (p.gb) store_elem<DT>(p.gb, j, b);
}

bool on_device(const tbe_layer_norm* h) {
    int d = -1;
    return cudaGetDevice(&d) == cudaSuccess && d == h->device;
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

template <int DT>
cudaError_t launch_forward(const NormForward& p, const tbe_layer_norm* h, cudaStream_t s) {
    norm_forward_kernel<DT><<<(unsigned)std::min<int64_t>(p.rows, h->num_sms * 8), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int DT>
cudaError_t launch_backward(const NormBackward& p, const tbe_layer_norm* h, cudaStream_t s) {
    if (p.gw || p.gb) norm_weight_kernel<DT><<<(p.D + kThreads - 1) / kThreads, kThreads, 0, s>>>(p);
    if (p.rows > 0)
        norm_backward_kernel<DT><<<(unsigned)std::min<int64_t>(p.rows, h->num_sms * 8), kThreads, 0, s>>>(p);
    return cudaGetLastError();
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
    return 256;
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
    const NormForward p{x, residual, weight, bias, x_stride, residual_stride, rows, h->c.dim, h->c.eps, out, total, stats};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = h->c.dtype == TBE_F32   ? launch_forward<DT_F32>(p, h, s)
                          : h->c.dtype == TBE_F16 ? launch_forward<DT_F16>(p, h, s)
                                                  : launch_forward<DT_BF16>(p, h, s);
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
    const NormBackward p{total, grad_out, grad_total, weight, total_stride, grad_out_stride, grad_total_stride, rows,
                         stats, h->c.dim, grad_x, grad_weight, grad_bias, static_cast<float*>(workspace)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = h->c.dtype == TBE_F32   ? launch_backward<DT_F32>(p, h, s)
                          : h->c.dtype == TBE_F16 ? launch_backward<DT_F16>(p, h, s)
                                                  : launch_backward<DT_BF16>(p, h, s);
    return e == cudaSuccess ? TBE_OK : cuda_fail(e);
}

}  // extern "C"
