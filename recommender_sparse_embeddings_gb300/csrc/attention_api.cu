// C ABI of the attention operators: argument checks, the handle, the
// workspaces' layout and the order of launches.  Declarations and contracts
// are in include/tbe.h.
#include <algorithm>
#include <new>
#include <utility>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "../../include/tbe.h"
#include "attention_mma.cuh"

namespace tbe {
int cuda_fail(cudaError_t e);
}

using namespace tbe;

struct tbe_attention {
    int device = 0;
    int num_sms = 0;
    AttnShape s{};
    void* dev = nullptr;
};

namespace {

struct CallRange {
    explicit CallRange(const char* name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange&) = delete;
    CallRange& operator=(const CallRange&) = delete;
};

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

int status(cudaError_t e) { return e == cudaSuccess ? TBE_OK : cuda_fail(e); }

bool on_device(const tbe_attention* h) {
    int d = -1;
    return cudaGetDevice(&d) == cudaSuccess && d == h->device;
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

bool vec_rows(const tbe_attention* h, const tbe_rows& r) {
    const int e = elem_bytes(h->s.dtype);
    return aligned16(r.data) && r.token_stride * e % 16 == 0 && r.head_stride * e % 16 == 0 && h->s.D * e % 16 == 0;
}

bool vec_pages(const tbe_attention* h, const tbe_pages& r) {
    const int e = elem_bytes(h->s.dtype);
    return aligned16(r.data) && r.page_stride * e % 16 == 0 && r.token_stride * e % 16 == 0 &&
           r.head_stride * e % 16 == 0 && h->s.D * e % 16 == 0;
}

bool rows_ok(const tbe_rows* r, int64_t n) {
    return r && (n == 0 || r->data) && r->token_stride >= 0 && r->head_stride >= 0;
}

bool pages_ok(const tbe_pages* r, int32_t num_pages) {
    return r && (num_pages == 0 || r->data) && r->page_stride >= 0 && r->token_stride >= 0 && r->head_stride >= 0;
}

// The tensor-core kernels take 16-bit rows of up to 128 columns that are
// 16-byte aligned; they hold tiles of 128 tokens.
constexpr int kMmaTile = 128;
bool takes_mma(const tbe_attention* h, bool vec) { return vec && h->s.dtype != TBE_F32 && h->s.D <= 128; }

Rows as_rows(const tbe_rows& r) { return Rows{r.data, r.token_stride, r.head_stride}; }

// The TMA map of a token operand, by the driver's encoder (found at run time;
// it computes 128 bytes on the host).  Of the two strides the larger has to be
// a multiple of the smaller, and neither 0: other layouts give false, and the
// call then takes the kernels that load by plain loads.
bool encode_rows(TileMap* map, const tbe_attention* h, const tbe_rows& r, int heads, int64_t N) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<Encode>(fn);
    }();
    if (!encode) return false;
    const int64_t token = r.token_stride, head = heads == 1 ? token : r.head_stride;
    map->heads_outer = head > token;
    const int64_t inner = std::min(token, head), outer = std::max(token, head);
    if (inner < h->s.D || outer % inner != 0 || outer >= (int64_t(1) << 38)) return false;
    cuuint64_t dims[3] = {(cuuint64_t)h->s.D, (cuuint64_t)heads, (cuuint64_t)N};
    cuuint32_t box[3] = {64, 1, 64};
    if (map->heads_outer) {
        std::swap(dims[1], dims[2]);
        std::swap(box[1], box[2]);
    }
    const cuuint64_t strides[2] = {(cuuint64_t)inner * 2, (cuuint64_t)outer * 2};
    const cuuint32_t steps[3] = {1, 1, 1};
    return encode(&map->map, h->s.dtype == TBE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                  const_cast<void*>(r.data), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool batch_within_limits(const tbe_attention* h, int64_t N, int64_t B) {
    if (N >= (int64_t(1) << 30) || B >= (int64_t(1) << 24)) return false;
    return ((N + 31) / 32 + B) * h->s.H < (int64_t(1) << 31);
}

int check_batch(const tbe_attention* h, const void* offsets, int32_t index_dtype, int64_t N, int32_t B) {
    if (!h || !on_device(h)) return TBE_ERR_INVALID_ARG;
    if (index_dtype != TBE_I32 && index_dtype != TBE_I64) return TBE_ERR_INVALID_ARG;
    if (N < 0 || B < 0 || !offsets || (B == 0 && N > 0)) return TBE_ERR_INVALID_ARG;
    return batch_within_limits(h, N, B) ? TBE_OK : TBE_ERR_UNSUPPORTED;
}

struct Layout {
    size_t n_items, items, delta, excess, size, bias_part, far_items, slot_of, far_part, total;
    int64_t capacity;
    FarWork far;  // sizes only
};

// How the first key tile's far queries are split (tensor-core backward): in
// chunks about as long as another tile's work, and of at least 32 blocks, so
// that N tokens make at most 2 N / (64 blocks) chunks and, with a slot for
// each split history's tile, half as many slots more.
FarWork far_split(const tbe_attention* h, int64_t N) {
    FarWork f{};
    if (h->s.sinks == 0 || h->s.window >= INT_MAX / 2 || h->s.dtype == TBE_F32 || h->s.D > 128) return f;
    f.near = (int32_t)((126 + (int64_t)h->s.window) / 64 + 1);
    f.blocks = std::max(32, h->s.window / 64 + 2);
    f.most = (int32_t)(2 * N / (64 * (int64_t)f.blocks));
    return f;
}

// Laid out for the smallest tile that any call of the handle takes, so that a
// workspace serves every smaller batch too.
Layout make_layout(const tbe_attention* h, int64_t N, int64_t B, bool backward) {
    Layout L{};
    L.capacity = N / (h->s.dtype == TBE_F32 || h->s.D > 128 ? 32 : 64) + B;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes);
        return at;
    };
    L.n_items = take(2 * sizeof(int32_t));  // of the tiles, of the far items
    L.items = take(sizeof(AttnItem) * (size_t)L.capacity);
    if (backward) {
        L.delta = take(sizeof(float) * (size_t)N * h->s.H);
        L.excess = take(sizeof(float) * (size_t)N * h->s.H);
        if (h->s.dtype == TBE_F16 && h->s.D <= 128) L.size = take(sizeof(float) * (size_t)N * h->s.H);
        L.far = far_split(h, N);
        L.bias_part = take(sizeof(float) * (size_t)(L.capacity + L.far.most) * h->s.H * h->s.buckets);
        if (L.far.most > 0) {
            L.far_items = take(sizeof(FarItem) * (size_t)L.far.most);
            L.slot_of = take(sizeof(int32_t) * (size_t)L.capacity);
            const size_t slots = (size_t)L.far.most + L.far.most / 2 + 1;
            L.far_part = take(sizeof(float) * slots * h->s.Hk * 2 * h->s.sinks * (h->s.D <= 64 ? 64 : 128));
        }
    }
    L.total = o;
    return L;
}

template <typename T>
T* at(void* base, size_t offset) {
    return reinterpret_cast<T*>(static_cast<char*>(base) + offset);
}

// The batch's work items: their source for the kernels, listed by a launch
// where there are many histories or some are split (or no kernel follows that
// would check the offsets).
int make_items(ItemSource* src, const tbe_attention* h, const Layout& L, const void* offsets, int32_t index_dtype,
               int64_t N, int32_t B, int tile, int64_t most, const FarWork& far, void* workspace, cudaStream_t s) {
    src->items = at<AttnItem>(workspace, L.items);
    src->n_items = at<int32_t>(workspace, L.n_items);
    src->offsets = B <= kScanHistories && far.most == 0 && N > 0 ? offsets : nullptr;
    src->index64 = index_dtype == TBE_I64;
    src->N = N;
    src->B = B;
    src->tile = tile;
    src->error = h->s.error;
    if (src->offsets) return TBE_OK;
    return status(launch_attn_items(offsets, src->index64, N, B, tile, at<AttnItem>(workspace, L.items), most,
                                    at<int32_t>(workspace, L.n_items), h->s.error, far, s));
}

// Rows of a cache that a query sees at most.
int64_t visible_most(const tbe_attention* h, int64_t max_length) {
    return std::min<int64_t>(max_length, (int64_t)h->s.window + h->s.sinks);
}

struct Split {
    int chunk, splits;
};

// CTAs that a decode call aims at, and those that one chunk makes.
int64_t decode_target(const tbe_attention* h) {
    return (int64_t)h->num_sms * (h->s.dtype == TBE_F32 || h->s.D > 128 ? 64 : 16);
}
int64_t decode_groups(const tbe_attention* h) {
    const int gt = attn_decode_heads(h->s.G);
    return (int64_t)h->s.Hk * ((h->s.G + gt - 1) / gt);
}

// Visible rows a decode CTA takes: small enough that the batch makes so many
// CTAs per SM that histories of uneven length leave no SM idle, and at least
// 256 (the join reads D + 2 floats per chunk and head, under 2 % of a chunk's
// rows).  The tensor-instruction kernel runs three CTAs per SM and pays about
// 3 us to start each: 16 (198 us for 128 bf16 histories of 4000 rows; 32: 205,
// 64: 215).  The FMA kernel is lighter: 64 (106 us for 200 fp32 histories of
// 600 rows; 32: 117, 16: 131).
Split decode_split(const tbe_attention* h, int64_t B, int64_t max_length) {
    const int64_t most = std::max<int64_t>(1, visible_most(h, max_length));
    const int64_t rows = std::max<int64_t>(1, B * decode_groups(h)), target = decode_target(h);
    int64_t chunk = (most * rows + target - 1) / target;
    chunk = std::max<int64_t>(256, (chunk + 63) / 64 * 64);
    if (most <= 512) chunk = std::max(chunk, most);  // not worth a second launch
    const int64_t splits = (most + chunk - 1) / chunk;
    return Split{(int)std::min<int64_t>(chunk, INT_MAX / 2), (int)splits};
}

// (history, chunk) pairs at most of any call of up to B histories and
// max_length tokens, so that a workspace serves smaller batches too.  Fewer
// histories make shorter chunks: b histories of m visible rows make at most
// b (1 + m / chunk) pairs, and a chunk holds at least 256 rows and at least
// m b groups / target.
int64_t decode_pairs(const tbe_attention* h, int64_t B, int64_t max_length) {
    const int64_t most = visible_most(h, max_length);
    if (most <= 512) return B;
    const int64_t target = decode_target(h), groups = decode_groups(h);
    return B + std::min(B * ((most + 255) / 256), (target + groups - 1) / groups);
}

}  // namespace

extern "C" {

int tbe_attention_create(const tbe_attention_config* c, tbe_attention** out) {
    CallRange range("tbe_attention_create");
    if (!out) return TBE_ERR_INVALID_ARG;
    *out = nullptr;
    if (!c) return TBE_ERR_INVALID_ARG;
    if (c->dtype != TBE_F32 && c->dtype != TBE_F16 && c->dtype != TBE_BF16) return TBE_ERR_INVALID_ARG;
    if (c->heads <= 0 || c->kv_heads <= 0 || c->heads % c->kv_heads != 0 || c->head_dim <= 0 || c->window < 0 ||
        c->sinks < 0 || c->num_buckets < 0 || !(c->scale > 0.f && c->scale - c->scale == 0.f))
        return TBE_ERR_INVALID_ARG;
    if (c->num_buckets > 0) {
        if (!c->bucket_starts || c->bucket_starts[0] != 0) return TBE_ERR_INVALID_ARG;
        if (c->num_buckets > kMaxBuckets) return TBE_ERR_UNSUPPORTED;
        for (int b = 1; b < c->num_buckets; ++b)
            if (c->bucket_starts[b] <= c->bucket_starts[b - 1]) return TBE_ERR_INVALID_ARG;
        if (c->bucket_starts[c->num_buckets - 1] > kMaxDistance) return TBE_ERR_UNSUPPORTED;
    }
    if (c->head_dim > kMaxHeadDim || c->sinks > kMaxSinks || c->heads > 1024) return TBE_ERR_UNSUPPORTED;

    tbe_attention* h = new (std::nothrow) tbe_attention();
    if (!h) return TBE_ERR_NO_MEMORY;
    AttnShape& s = h->s;
    s.dtype = c->dtype;
    s.H = c->heads;
    s.Hk = c->kv_heads;
    s.G = c->heads / c->kv_heads;
    s.D = c->head_dim;
    s.window = c->window == 0 ? INT_MAX / 2 : std::min(c->window, INT_MAX / 2);
    s.sinks = c->sinks;
    s.buckets = c->num_buckets;
    s.scale = c->scale;
    s.far = s.buckets > 0 ? c->bucket_starts[s.buckets - 1] : 0;
    int optin = 0;
    cudaError_t e = cudaGetDevice(&h->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, h->device);
    if (e == cudaSuccess) e = attn_simt_configure(optin);
    if (e == cudaSuccess) e = attn_forward_mma_configure();
    if (e == cudaSuccess) e = attn_backward_mma_configure();
    if (e != cudaSuccess) {
        delete h;
        return cuda_fail(e);
    }
    // device block: the error word, the buckets' first distances (one more,
    // INT_MAX, ends the last), the bucket of every distance up to `far`
    const size_t starts_at = sizeof(AttnBlock), map_at = starts_at + sizeof(int32_t) * (s.buckets + 1);
    const size_t bytes = map_at + sizeof(uint16_t) * (s.far + 1);
    try {
        std::vector<unsigned char> img(bytes, 0);
        int32_t* starts = reinterpret_cast<int32_t*>(img.data() + starts_at);
        uint16_t* map = reinterpret_cast<uint16_t*>(img.data() + map_at);
        for (int b = 0; b < s.buckets; ++b) starts[b] = c->bucket_starts[b];
        starts[s.buckets] = INT_MAX;
        for (int d = 0, b = 0; s.buckets > 0 && d <= s.far; ++d) {
            while (starts[b + 1] <= d) ++b;
            map[d] = (uint16_t)b;
        }
        e = cudaMalloc(&h->dev, bytes);
        if (e == cudaSuccess) e = cudaMemcpy(h->dev, img.data(), bytes, cudaMemcpyHostToDevice);
    } catch (const std::bad_alloc&) {
        delete h;
        return TBE_ERR_NO_MEMORY;
    }
    if (e != cudaSuccess) {
        if (h->dev) cudaFree(h->dev);
        delete h;
        return e == cudaErrorMemoryAllocation ? TBE_ERR_NO_MEMORY : cuda_fail(e);
    }
    s.error = &static_cast<AttnBlock*>(h->dev)->error;
    s.starts = at<int32_t>(h->dev, starts_at);
    s.bucket_of = at<uint16_t>(h->dev, map_at);
    *out = h;
    return TBE_OK;
}

void tbe_attention_destroy(tbe_attention* h) {
    if (!h) return;
    if (h->dev) cudaFree(h->dev);
    delete h;
}

size_t tbe_attention_workspace_bytes(const tbe_attention* h, int64_t N, int32_t B, int32_t backward) {
    if (!h || N < 0 || B < 0 || !batch_within_limits(h, N, B)) return 0;
    return make_layout(h, N, B, backward != 0).total;
}

int tbe_attention_forward(tbe_attention* h, const tbe_rows* q, const tbe_rows* k, const tbe_rows* v, const void* bias,
                          const void* offsets, int32_t index_dtype, int64_t N, int32_t B, void* out, float* lse,
                          void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range("tbe_attention_forward");
    int rc = check_batch(h, offsets, index_dtype, N, B);
    if (rc) return rc;
    if (!rows_ok(q, N) || !rows_ok(k, N) || !rows_ok(v, N)) return TBE_ERR_INVALID_ARG;
    if ((bias != nullptr) != (h->s.buckets > 0) || (N > 0 && (!out || !lse)) || !workspace || !aligned16(workspace))
        return TBE_ERR_INVALID_ARG;
    const Layout L = make_layout(h, N, B, false);
    if (workspace_bytes < L.total) return TBE_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    AttnForward p{};
    p.s = h->s;
    p.q = as_rows(*q);
    p.k = as_rows(*k);
    p.v = as_rows(*v);
    p.bias = bias;
    p.out = out;
    p.lse = lse;
    p.N = N;
    p.vec = vec_rows(h, *q) && vec_rows(h, *k) && vec_rows(h, *v) && aligned16(out);
    AttnMaps maps{};
    const bool mma = N > 0 && takes_mma(h, p.vec) && encode_rows(&maps.q, h, *q, h->s.H, N) &&
                     encode_rows(&maps.k, h, *k, h->s.Hk, N) && encode_rows(&maps.v, h, *v, h->s.Hk, N);
    const int tile = mma ? kMmaTile : attn_simt_tile(h->s.dtype, h->s.D, h->s.H, N, B, h->num_sms);
    const int64_t most = N / tile + B;
    rc = make_items(&p.src, h, L, offsets, index_dtype, N, B, tile, most, FarWork{}, workspace, s);
    if (rc || N == 0) return rc;
    // tiles in turn: where they are listed (there are many) and a token sees few
    // keys, so that a tile's start and end are most of it.  Long tiles are handed
    // out better one by one, as others end.  bf16, us in turn / each by itself:
    //   512 histories of 150 tokens, 4 heads of 64, all visible   91 / 100
    //   256 of 1500, window 128                                  398 / 422
    //   160 of 500, all visible, 4 heads (16 heads)              130 / 117 (398 / 408)
    //   160 of 1500, all visible                                 635 / 526
    p.max_items = most;
    const int64_t sees = std::min(N / B, (int64_t)h->s.window + h->s.sinks);
    p.ctas = !p.src.offsets && sees <= 256 ? 2 * h->num_sms : 0;
    return status(mma ? launch_attn_forward_mma(p, maps, s) : launch_attn_forward_simt(p, most, s));
}

int tbe_attention_backward(tbe_attention* h, const tbe_rows* q, const tbe_rows* k, const tbe_rows* v, const void* bias,
                           const void* offsets, int32_t index_dtype, int64_t N, int32_t B, const void* out,
                           const float* lse, const tbe_rows* grad_out, void* grad_q, void* grad_k, void* grad_v,
                           void* grad_bias, void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range("tbe_attention_backward");
    int rc = check_batch(h, offsets, index_dtype, N, B);
    if (rc) return rc;
    if (!rows_ok(q, N) || !rows_ok(k, N) || !rows_ok(v, N) || !rows_ok(grad_out, N)) return TBE_ERR_INVALID_ARG;
    if ((bias != nullptr) != (h->s.buckets > 0) || (grad_bias != nullptr) != (h->s.buckets > 0) || !workspace ||
        !aligned16(workspace))
        return TBE_ERR_INVALID_ARG;
    if (N > 0 && (!out || !lse || !grad_q || !grad_k || !grad_v)) return TBE_ERR_INVALID_ARG;
    const Layout L = make_layout(h, N, B, true);
    if (workspace_bytes < L.total) return TBE_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    AttnBackward p{};
    p.s = h->s;
    p.q = as_rows(*q);
    p.k = as_rows(*k);
    p.v = as_rows(*v);
    p.g = as_rows(*grad_out);
    p.bias = bias;
    p.out = out;
    p.lse = lse;
    p.gq = grad_q;
    p.gk = grad_k;
    p.gv = grad_v;
    p.delta = at<float>(workspace, L.delta);
    p.excess = at<float>(workspace, L.excess);
    p.size = at<float>(workspace, L.size);
    p.bias_part = at<float>(workspace, L.bias_part);
    p.N = N;
    p.vec = vec_rows(h, *q) && vec_rows(h, *k) && vec_rows(h, *v) && vec_rows(h, *grad_out) && aligned16(out) &&
            aligned16(grad_q) && aligned16(grad_k) && aligned16(grad_v);
    AttnMaps maps{};
    const bool mma = N > 0 && takes_mma(h, p.vec) && encode_rows(&maps.q, h, *q, h->s.H, N) &&
                     encode_rows(&maps.k, h, *k, h->s.Hk, N) && encode_rows(&maps.v, h, *v, h->s.Hk, N) &&
                     encode_rows(&maps.g, h, *grad_out, h->s.H, N);
    const int tile = mma ? kMmaTile : attn_simt_tile(h->s.dtype, h->s.D, h->s.H, N, B, h->num_sms);
    const int64_t most = N / tile + B;
    p.max_items = most;
    if (mma && L.far.most > 0) {
        p.far = L.far;
        p.far.items = at<FarItem>(workspace, L.far_items);
        p.far.n_items = at<int32_t>(workspace, L.n_items) + 1;
        p.far.slot_of = at<int32_t>(workspace, L.slot_of);
        p.far.part = at<float>(workspace, L.far_part);
    }
    rc = make_items(&p.src, h, L, offsets, index_dtype, N, B, tile, most, p.far, workspace, s);
    if (rc) return rc;
    if (N > 0) rc = status(mma ? launch_attn_backward_mma(p, maps, most, s) : launch_attn_backward_simt(p, most, s));
    if (rc || !bias) return rc;
    return status(launch_attn_bias_reduce(p, grad_bias, s));
}

int tbe_attention_append(tbe_attention* h, const tbe_rows* k, const tbe_rows* v, const void* offsets,
                         int32_t index_dtype, int64_t N, int32_t B, const int32_t* before, const tbe_pages* k_pages,
                         const tbe_pages* v_pages, int32_t num_pages, int32_t page_size, const int32_t* block_table,
                         int32_t table_width, void* stream) {
    CallRange range("tbe_attention_append");
    const int rc = check_batch(h, offsets, index_dtype, N, B);
    if (rc) return rc;
    if (!rows_ok(k, N) || !rows_ok(v, N)) return TBE_ERR_INVALID_ARG;
    if (!pages_ok(k_pages, num_pages) || !pages_ok(v_pages, num_pages)) return TBE_ERR_INVALID_ARG;
    if (num_pages < 0 || page_size <= 0 || table_width < 0 || (B > 0 && (!before || (table_width > 0 && !block_table))))
        return TBE_ERR_INVALID_ARG;
    if ((int64_t)table_width * page_size >= (int64_t(1) << 30)) return TBE_ERR_UNSUPPORTED;
    if (N == 0) return TBE_OK;
    AttnAppend p{};
    p.Hk = h->s.Hk;
    p.D = h->s.D;
    p.e = elem_bytes(h->s.dtype);
    p.k = as_rows(*k);
    p.v = as_rows(*v);
    p.offsets = offsets;
    p.index64 = index_dtype == TBE_I64;
    p.before = before;
    p.kp = k_pages->data;
    p.vp = v_pages->data;
    p.k_page = k_pages->page_stride;
    p.k_token = k_pages->token_stride;
    p.k_head = k_pages->head_stride;
    p.v_page = v_pages->page_stride;
    p.v_token = v_pages->token_stride;
    p.v_head = v_pages->head_stride;
    p.table = block_table;
    p.width = table_width;
    p.num_pages = num_pages;
    p.B = B;
    p.N = N;
    p.page = make_fast_div((uint32_t)page_size);
    p.error = h->s.error;
    p.vec = vec_rows(h, *k) && vec_rows(h, *v) && vec_pages(h, *k_pages) && vec_pages(h, *v_pages);
    return status(launch_attn_append(p, static_cast<cudaStream_t>(stream)));
}

size_t tbe_attention_decode_workspace_bytes(const tbe_attention* h, int32_t B, int64_t max_length) {
    if (!h || B < 0 || B >= (1 << 24) || max_length < 0 || max_length >= (int64_t(1) << 30)) return 0;
    return align_up(sizeof(float) * (size_t)decode_pairs(h, B, max_length) * h->s.H * (h->s.D + 2)) + 256;
}

int tbe_attention_decode(tbe_attention* h, const tbe_rows* q, const tbe_pages* k_pages, const tbe_pages* v_pages,
                         int32_t num_pages, int32_t page_size, const int32_t* block_table, int32_t table_width,
                         const int32_t* lengths, int32_t B, int64_t max_length, const void* bias, void* out,
                         void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range("tbe_attention_decode");
    if (!h || !on_device(h)) return TBE_ERR_INVALID_ARG;
    if (B < 0 || max_length < 0 || num_pages < 0 || page_size <= 0 || table_width < 0) return TBE_ERR_INVALID_ARG;
    if (!rows_ok(q, B) || !pages_ok(k_pages, num_pages) || !pages_ok(v_pages, num_pages)) return TBE_ERR_INVALID_ARG;
    if ((bias != nullptr) != (h->s.buckets > 0) || !workspace || !aligned16(workspace)) return TBE_ERR_INVALID_ARG;
    if (B > 0 && (!lengths || !out || (table_width > 0 && !block_table))) return TBE_ERR_INVALID_ARG;
    if ((int64_t)table_width * page_size >= (int64_t(1) << 30) || B >= (1 << 24)) return TBE_ERR_UNSUPPORTED;
    const int64_t room = (int64_t)table_width * page_size;
    const int64_t most = max_length == 0 ? room : std::min(max_length, room);
    const Split sp = decode_split(h, B, most);
    const int gt = attn_decode_heads(h->s.G);
    if ((int64_t)sp.splits * ((h->s.G + gt - 1) / gt) * h->s.Hk * B >= (int64_t(1) << 31) ||
        (int64_t)B * h->s.H >= (int64_t(1) << 31))
        return TBE_ERR_UNSUPPORTED;
    if (workspace_bytes < sizeof(float) * (size_t)B * h->s.H * sp.splits * (h->s.D + 2))
        return TBE_ERR_WORKSPACE_TOO_SMALL;
    if (B == 0) return TBE_OK;
    AttnDecode p{};
    p.s = h->s;
    p.q = as_rows(*q);
    p.kp = k_pages->data;
    p.vp = v_pages->data;
    p.k_page = k_pages->page_stride;
    p.k_token = k_pages->token_stride;
    p.k_head = k_pages->head_stride;
    p.v_page = v_pages->page_stride;
    p.v_token = v_pages->token_stride;
    p.v_head = v_pages->head_stride;
    p.table = block_table;
    p.lengths = lengths;
    p.bias = bias;
    p.out = out;
    p.part = static_cast<float*>(workspace);
    p.width = table_width;
    p.num_pages = num_pages;
    p.B = B;
    p.chunk = sp.chunk;
    p.splits = sp.splits;
    p.max_length = most;
    p.page = make_fast_div((uint32_t)page_size);
    p.vec = vec_rows(h, *q) && vec_pages(h, *k_pages) && vec_pages(h, *v_pages);
    return status(launch_attn_decode(p, static_cast<cudaStream_t>(stream)));
}

int tbe_attention_get_error(tbe_attention* h, void* stream) {
    if (!h || !on_device(h)) return TBE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t bits = 0;
    cudaError_t e = cudaMemcpyAsync(&bits, h->s.error, sizeof bits, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = cudaMemsetAsync(h->s.error, 0, sizeof(uint32_t), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e);
    if (bits & ERR_TIMEOUT) return TBE_ERR_TIMEOUT;
    if (bits & ERR_OFFSETS) return TBE_ERR_BAD_OFFSETS;
    if (bits & ERR_OOB) return TBE_ERR_INDEX_OOB;
    return TBE_OK;
}

}  // extern "C"
