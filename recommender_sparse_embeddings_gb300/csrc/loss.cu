// Softmax cross entropy of rows over a table of items, and its gradients.
// Declarations, formulas and contracts are in include/tbe.h.
#include <algorithm>
#include <mutex>
#include <new>

#include <nvtx3/nvToolsExt.h>

#include "../../include/tbe.h"
#include "loss_mma.cuh"

namespace tbe {
int cuda_fail(cudaError_t e);
}

using namespace tbe;

struct tbe_softmax_loss {
    int device = 0;
    int num_sms = 0;
    tbe_softmax_loss_config c{};
    uint32_t* error = nullptr;
    // the last sizes' slices (the choice takes the host 5 us, as long as a launch).
    // Under a lock: workspaces are laid out for the slices of their own sizes, so a
    // handle used from two host threads against the rules must not mix them up.
    mutable std::mutex choice_mu;
    mutable struct {
        int64_t rows = -1, items = -1;
        int slices;
    } forward_choice;
    mutable struct {
        int64_t rows = -1, items = -1;
        int x, w;
    } backward_choice;
};

namespace {

constexpr int kMaxLossDim = 4096;

struct CallRange {
    explicit CallRange(const char* name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange&) = delete;
    CallRange& operator=(const CallRange&) = delete;
};

// Rows of a 16-bit operand: P planes of [rows][pitch].
struct Copy {
    const void* from;
    int64_t stride, rows;
    int32_t D, pitch;
    uint16_t* to;
    bool vec;
};

template <int DT>
__device__ __forceinline__ void copy_row(const Copy& c, int64_t row, bool zero, int lane) {
    const int64_t in = row * c.stride, out = row * c.pitch, plane = c.rows * c.pitch;
    if constexpr (DT == DT_F32) {
        for (int j = lane; j < c.D; j += 32) {
            float x = zero ? 0.f : load_elem<DT>(c.from, in + j);
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                const __nv_bfloat16 y = __float2bfloat16_rn(x);
                x -= __bfloat162float(y);
                c.to[p * plane + out + j] = __bfloat16_as_ushort(y);
            }
        }
    } else if (c.vec) {
        for (int j = lane; j < c.D / 8; j += 32)
            reinterpret_cast<uint4*>(c.to + out)[j] =
                zero ? make_uint4(0, 0, 0, 0)
                     : __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(c.from) + in) + j);
    } else {
        for (int j = lane; j < c.D; j += 32)
            c.to[out + j] = zero ? (uint16_t)0 : __ldg(static_cast<const uint16_t*>(c.from) + in + j);
    }
}

// One warp a row.
template <int DT>
__global__ void __launch_bounds__(256) loss_copy_kernel(const Copy c) {
    chain_wait();
    for (int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 32; row < c.rows; row += (int64_t)gridDim.x * 8)
        copy_row<DT>(c, row, false, threadIdx.x % 32);
}

struct RowsIn {
    Copy x;
    const void* targets;
    int32_t index64, parts;  // parts: of gmax; 0: each CTA looks through the rows by itself
    int64_t V, tiles;
    const float *lse, *g;
    float scale;
    float* rows;  // [tiles][kRowValues]
    float* unit;  // what the products of d are multiplied by
    float* gmax;  // [kMaxCtas] partial maxima
    uint32_t* error;
};

__device__ __forceinline__ int64_t row_target(const RowsIn& p, int64_t row) {
    const int64_t t =
        p.index64 ? static_cast<const int64_t*>(p.targets)[row] : static_cast<const int32_t*>(p.targets)[row];
    if (t >= p.V) atomicOr(p.error, ERR_OOB);
    return t >= 0 && t < p.V ? t : -1;
}

// The largest finite |g scale| of the rows from `first` on, in steps.
__device__ __forceinline__ float row_max(const RowsIn& p, int64_t first, int64_t step) {
    __shared__ float most[8];
    float m = 0.f;
    for (int64_t row = first; row < p.x.rows; row += step) {
        const float a = fabsf(p.g[row] * p.scale);
        if (a <= FLT_MAX && row_target(p, row) >= 0) m = fmaxf(m, a);
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (threadIdx.x % 32 == 0) most[threadIdx.x / 32] = m;
    __syncthreads();
    for (int w = 0; w < 8; ++w) m = fmaxf(m, most[w]);
    return m;
}

// It in parts, where there are many rows.
constexpr int kMaxCtas = 64, kFewRows = 2048;
__global__ void __launch_bounds__(256) loss_max_kernel(const RowsIn p) {
    chain_wait();
    const float m = row_max(p, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
    if (threadIdx.x == 0) p.gmax[blockIdx.x] = m;
}

// The backward pass's rows, one warp each: x copied with zeros in the rows left
// out, and what each row brings.
//
// The fused kernel's grad_x sums p - [target] and multiplies the row's sum by its own
// g.  In sums over the rows (and in the step kernel, whose d serves both gradients) d
// is held relative to the largest |g scale|.  So where all rows have the same g (a
// mean), d is p - [target] itself: nothing has to be multiplied, and -1 for a
// target of little weight has no rounding, where -g would be off by the same 2^-9
// in every row (grad_table of 300 rows over 5000 items in bf16: 0.0025 off, so
// 0.0017).  fp16's range is narrow besides (6e-8 to 65504): there d comes times
// target_unit = 2^14, and weights down to 2^-28 keep all their bits.
template <int DT>
__global__ void __launch_bounds__(256) loss_rows_kernel(const RowsIn p) {
    chain_wait();
    const int lane = threadIdx.x % 32;
    float m = 0.f;
    if (p.parts == 0) {
        m = row_max(p, threadIdx.x, 256);
    } else {
        m = fmaxf(p.gmax[lane], p.gmax[lane + 32]);
#pragma unroll
        for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if (!(m > 0.f)) m = 1.f;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.unit = m / target_unit<DT>();
    for (int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 32; row < p.tiles * 128;
         row += (int64_t)gridDim.x * 8) {
        float* to = p.rows + row / 128 * kRowValues + row % 128;
        const int64_t t = row < p.x.rows ? row_target(p, row) : -1;
        if (row < p.x.rows) copy_row<DT>(p.x, row, t < 0, lane);
        if (lane == 0) {
            to[0] = t < 0 ? -INFINITY : DT == DT_F32 ? -p.lse[row] : log2f(target_unit<DT>()) - p.lse[row] * kLog2e;
            to[128] = t < 0 ? 1.f : p.g[row] * p.scale / m;
            to[256] = __int_as_float((int)t);
            to[384] = t < 0 ? 0.f : p.g[row] * p.scale / target_unit<DT>();
        }
    }
}

// The slices' sums of a row joined, by one warp.
template <int DT>
__global__ void __launch_bounds__(256)
    loss_join_kernel(const float2* part, int parts, const float* picked, const void* targets, int index64, int64_t N,
                     int64_t V, float* loss, float* lse) {
    chain_wait();
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 32;
    const int lane = threadIdx.x % 32;
    if (row >= N) return;
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, part[row * parts + i].x);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
    for (int i = lane; i < parts; i += 32) {
        const float2 y = part[row * parts + i];
        // (a part that no item reaches: -inf and 0)
        if (!(y.y == 0.f)) l = fmaf(y.y, ex2(DT == DT_F32 ? (y.x - m) * kLog2e : y.x - m), l);
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane != 0) return;
    const int64_t t = index64 ? static_cast<const int64_t*>(targets)[row] : static_cast<const int32_t*>(targets)[row];
    constexpr float kNatural = DT == DT_F32 ? 1.f : 0.6931471805599453f;
    const float log_l = logf(l);
    lse[row] = fmaf(m, kNatural, log_l);
    loss[row] = t >= 0 && t < V ? fmaf(m - picked[row], kNatural, log_l) : 0.f;
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

// ---- workspaces and plans

template <typename T>
T* at(void* base, size_t offset) {
    return reinterpret_cast<T*>(static_cast<char*>(base) + offset);
}

int64_t up_to(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Bytes of a piece of d (per plane of fp32's three).  Long pieces make few
// launches, each with a start and an end in which SMs idle; shorter ones would
// stay in L2 (129 MB), which gains less.  Pieces of 48, 64, 96 and 150 MB: 4096 x
// 32768 x 512 bf16 473, 442, 379 and 369 us, 8192 x 20000 x 256 fp32 1733, 1537, 1384
// and 1426, 2048 x 30000 x 4096 bf16 1215, 1174, 1269 and 1380.
constexpr int64_t kPieceBytes = 96 << 20;
// Work items that the sums' parts make at most: four a SM of the 152, as many and
// as few as even out (forward 8192 x 131072 x 256 bf16 338 us; 304 items 387, 1216 337,
// with twice the room).  The slices tried below are a few small numbers and the SMs'
// count, its half and multiples; a GPU of other counts would be served, less evenly.
constexpr int kMostParts = 608;
constexpr int kRowCtas = 1024;

struct Plan {
    int planes, pitch, cols4, col_tiles;
    int64_t row_tiles;
    int64_t piece;  // items
    int64_t span;   // items of a copied part of the table, whole pieces
    size_t rows, unit, x, w, d, x_part, w_part, total;  // offsets
    size_t w_bytes, d_bytes, w_part_bytes;              // of one of two
};

// What a product is multiplied by on its way into the softmax.
float argument_scale(const tbe_softmax_loss* h) { return h->c.dtype == TBE_F32 ? h->c.scale : h->c.scale * kLog2e; }

// Whether the fused kernel takes the call (its sums are up to 256 columns wide,
// and of fp32's three planes 128 columns fill shared memory); others go through
// pieces of d in memory.
bool takes_fused(const tbe_softmax_loss* h) { return h->c.dim <= (h->c.dtype == TBE_F32 ? 128 : 256); }

// Sized so that a workspace serves every smaller call: each size grows with N
// and V although the piece shrinks with N.
Plan make_plan(const tbe_softmax_loss* h, int64_t N, int64_t V, bool backward, bool copied) {
    Plan L{};
    const bool fused = backward && takes_fused(h);
    const int D = h->c.dim;
    L.planes = h->c.dtype == TBE_F32 ? 3 : 1;
    L.pitch = (int)up_to(D, 8);
    L.cols4 = (int)up_to(D, 32) / 4;
    L.col_tiles = (D + 255) / 256;
    L.row_tiles = (N + 127) / 128;
    const int64_t padded = up_to(V, 256), room = kPieceBytes / (2 * L.planes);  // elements
    L.piece = std::max<int64_t>(256, std::min(padded, room / std::max<int64_t>(N, 1) / 256 * 256));
    const int64_t item_bytes = 2 * (int64_t)L.planes * L.pitch;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t here = o;
        o = align_up(o + bytes);
        return here;
    };
    L.x = take((size_t)N * item_bytes);
    if (copied) {
        // 16-bit tables of aligned rows are read where they are; a copy is rare
        const int64_t budget = h->c.dtype != TBE_F32 && D % 8 == 0 ? 16 << 20 : 64 << 20;
        const int64_t items = std::max<int64_t>(256, budget / item_bytes / 256 * 256);
        L.piece = std::min(L.piece, items);
        L.span = backward && !fused ? items / L.piece * L.piece : items;
        L.w_bytes = align_up((size_t)(std::min(padded, items) * item_bytes));
        L.w = take(2 * L.w_bytes);
    }
    if (backward) {
        L.rows = take(sizeof(float) * kRowValues * L.row_tiles);
        L.unit = take(sizeof(float) * (1 + kMaxCtas));
        const size_t tile = (size_t)L.cols4 * 128 * sizeof(float4);
        // (one sum over all items needs no slabs, and several make kMostParts tiles at most)
        L.x_part = take(std::max<int64_t>(L.row_tiles, kMostParts / L.col_tiles + 1) * tile);
        // (the fused kernel's long sums of 16-bit types over the rows: a slab of each tile of items)
        const int64_t long_tiles =
            fused && L.planes == 1 && N > kLongSum ? (copied ? std::min(padded, L.span) : padded) / 128 : 0;
        L.w_part_bytes = (size_t)std::max<int64_t>(kMostParts / L.col_tiles + 1, long_tiles) * tile;
        L.w_part = take((fused ? 1 : 2) * L.w_part_bytes);
        if (!fused) {
            L.d_bytes = align_up((size_t)std::min(std::max(room, 256 * N), N * padded) * 2 * L.planes);
            L.d = take(2 * L.d_bytes);
        }
    } else {
        L.rows = take(sizeof(float) * N);                                   // picked
        L.d = take(sizeof(float2) * 4 * (N + 128 * (int64_t)kMostParts));  // part
    }
    L.total = o + 256;
    return L;
}

// A map of 16-bit rows: (column, row, plane), boxes of 64 columns x `box` rows
// in the 128-byte swizzle; zeros outside.  The encoder is the driver's, found at
// run time (it computes 128 bytes on the host).
bool encode(CUtensorMap* map, int dtype, const void* base, int64_t D, int64_t rows, int planes, int64_t pitch, int box) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)pitch * 2 * (planes > 1 ? rows : 1)};
    const cuuint32_t boxes[3] = {64, (cuuint32_t)box, 1}, steps[3] = {1, 1, 1};
    return fn(map, dtype == TBE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
              const_cast<void*>(base), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether TMA reads these rows where they are.
bool direct(const tbe_softmax_loss* h, const void* p, int64_t stride, int64_t rows) {
    return h->c.dtype != TBE_F32 && aligned16(p) &&
           (rows == 1 ? h->c.dim % 8 == 0 : stride % 8 == 0 && stride >= h->c.dim) && stride < (int64_t(1) << 38);
}

Copy make_copy(const tbe_softmax_loss* h, const void* from, int64_t stride, int64_t rows, int pitch, void* to) {
    return Copy{from, stride, rows, h->c.dim, pitch, static_cast<uint16_t*>(to),
                aligned16(from) && stride % 8 == 0 && h->c.dim % 8 == 0};
}

cudaError_t launch_copy(const tbe_softmax_loss* h, const Copy& c, cudaStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>((c.rows + 7) / 8, (int64_t)h->num_sms * 16);
    return h->c.dtype == TBE_F32 ? launch_chained(loss_copy_kernel<DT_F32>, dim3(grid), dim3(256), s, c)
                                 : launch_chained(loss_copy_kernel<DT_F16>, dim3(grid), dim3(256), s, c);
}

// The table's maps over the pieces of a call: the table itself, or spans of it
// copied in turn into one of two places.
struct Table {
    const tbe_softmax_loss* h;
    const void* data;
    int64_t stride, V, span;
    int planes, pitch;
    bool is_direct;
    char* room;
    size_t room_bytes;
    int64_t now = -1;

    int64_t first(int64_t item) const { return is_direct ? 0 : item / span * span; }

    bool map(CUtensorMap* m, int64_t item) const {
        if (is_direct)
            return encode(m, h->c.dtype, data, h->c.dim, V, 1, V == 1 ? pitch : stride, 64);
        const int64_t k = item / span, rows = std::min(span, V - k * span);
        return encode(m, h->c.dtype, room + (k & 1) * room_bytes, h->c.dim, rows, planes, pitch, 64);
    }
    // Copies the item's span unless that was done.
    cudaError_t fetch(int64_t item, cudaStream_t s) {
        if (is_direct || item / span == now) return cudaSuccess;
        now = item / span;
        const int64_t from = now * span;
        return launch_copy(h,
                           make_copy(h, static_cast<const char*>(data) + from * stride * elem_bytes(h->c.dtype), stride,
                                     std::min(span, V - from), pitch, room + (now & 1) * room_bytes),
                           s);
    }
};

// Slices of the table a row tile's items are cut into: those that end soonest
// with every CTA taking items in turn.
int choose_slices(int64_t row_tiles, int64_t item_tiles, int ctas) {
    int best = 1;
    int64_t least = INT64_MAX;
    const int64_t most = std::min<int64_t>(item_tiles, std::max<int64_t>(1, kMostParts / row_tiles));
    for (int64_t s = 1; s <= most; ++s) {
        const int64_t turns = (row_tiles * s + ctas - 1) / ctas, time = turns * ((item_tiles + s - 1) / s);
        if (time < least) {
            least = time;
            best = (int)s;
        }
    }
    return best;
}

int forward(const tbe_softmax_loss* h, const Plan& L, LossForward p, const void* x, int64_t x_stride, const void* table,
            int64_t table_stride, float* loss, float* lse, char* base, cudaStream_t s) {
    LossMaps maps{};
    const bool as_is = direct(h, x, x_stride, p.N);
    cudaError_t e = cudaSuccess;
    if (!as_is) e = launch_copy(h, make_copy(h, x, x_stride, p.N, L.pitch, base + L.x), s);
    if (e != cudaSuccess) return cuda_fail(e);
    if (!encode(&maps.x, h->c.dtype, as_is ? x : base + L.x, p.D, p.N, L.planes,
                as_is && p.N > 1 ? x_stride : L.pitch, 64))
        return TBE_ERR_CUDA;
    Table w{h, table, table_stride, p.V, L.span, L.planes, L.pitch, direct(h, table, table_stride, p.V), base + L.w,
            L.w_bytes};
    const int64_t whole = w.is_direct ? p.V : std::min(p.V, L.span);
    p.row_tiles = (int)L.row_tiles;
    {
        std::lock_guard<std::mutex> lock(h->choice_mu);
        auto& last = h->forward_choice;
        if (last.rows != L.row_tiles || last.items != whole) {
            last.slices = choose_slices(L.row_tiles, (whole + 255) / 256, h->num_sms);
            last.rows = L.row_tiles;
            last.items = whole;
        }
        p.slices = last.slices;
    }
    p.part = at<float2>(base, L.d);
    p.picked = at<float>(base, L.rows);
    for (p.v0 = 0; p.v0 < p.V; p.v0 = p.v1) {
        p.v1 = std::min(p.V, p.v0 + whole);
        p.w0 = w.first(p.v0);
        p.first = p.v0 == 0;
        p.item_tiles = (int)((p.v1 - p.v0 + 255) / 256);
        e = w.fetch(p.v0, s);
        if (e != cudaSuccess) return cuda_fail(e);
        if (!w.map(&maps.w, p.v0)) return TBE_ERR_CUDA;
        const int64_t items = (int64_t)p.row_tiles * p.slices;
        e = launch_loss_forward(p, maps, h->c.dtype, (int)std::min<int64_t>(items, h->num_sms), s);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    auto* join = h->c.dtype == TBE_F32 ? loss_join_kernel<DT_F32> : loss_join_kernel<DT_BF16>;
    return status(launch_chained(join, dim3((unsigned)((p.N + 7) / 8)), dim3(256), s,
                                 (const float2*)p.part, 4 * p.slices, (const float*)p.picked, p.targets, p.index64, p.N,
                                 p.V, loss, lse));
}

cudaError_t launch_rows(const tbe_softmax_loss* h, const Plan& L, RowsIn rows, char* base, cudaStream_t s) {
    rows.rows = at<float>(base, L.rows);
    rows.unit = at<float>(base, L.unit);
    rows.gmax = rows.unit + 1;
    rows.tiles = L.row_tiles;
    rows.x.to = at<uint16_t>(base, L.x);
    const dim3 grid((unsigned)std::min<int64_t>(rows.tiles * 16, kRowCtas));
    rows.parts = rows.x.rows > kFewRows ? kMaxCtas : 0;
    if (rows.parts > 0) {
        const cudaError_t e = launch_chained(loss_max_kernel, dim3(kMaxCtas), dim3(256), s, rows);
        if (e != cudaSuccess) return e;
    }
    return h->c.dtype == TBE_F32   ? launch_chained(loss_rows_kernel<DT_F32>, grid, dim3(256), s, rows)
           : h->c.dtype == TBE_F16 ? launch_chained(loss_rows_kernel<DT_F16>, grid, dim3(256), s, rows)
                                   : launch_chained(loss_rows_kernel<DT_BF16>, grid, dim3(256), s, rows);
}

// Slices of the fused launch's sums, x's and w's: those of the least estimated
// time, in units of one walked tile (0.35 to 0.7 us).  A CTA's start and end take
// about 4 of them, a slab's way through memory one per 64 columns; more CTAs than
// SMs share the work evenly but for about half of one at the end.
void choose_sides(LossSide* x, LossSide* w, int D, int ctas) {
    static constexpr int kTry[] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 16, 24, 32, 48, 76, 152, 304, 608};
    double least = 1e300;
    LossSide a = *x, b = *w;
    auto cost = [&](const LossSide& s) {
        return (s.others + s.slices - 1) / s.slices + 4 + (s.slices > 1 ? (D + 63) / 64 : 0);
    };
    auto allowed = [](const LossSide& s, int slices) {
        return slices == 1 || (slices <= s.others && (int64_t)slices * s.tiles <= kMostParts);
    };
    for (int i : kTry) {
        if (!allowed(*x, i)) continue;
        a.slices = i;
        const int ca = cost(a);
        for (int j : kTry) {
            if (!allowed(*w, j)) continue;
            b.slices = j;
            const int cb = cost(b);
            const int64_t na = (int64_t)x->tiles * i, nb = (int64_t)w->tiles * j, n = na + nb;
            double time = std::max(ca, cb);
            if (n > ctas)
                time = std::max(time, ((double)na * ca + (double)nb * cb) / ctas + 0.5 * cb);
            if (time < least) {
                least = time;
                x->slices = i;
                w->slices = j;
            }
        }
    }
}

int backward_fused(const tbe_softmax_loss* h, const Plan& L, LossFused p, const RowsIn& rows, const void* table,
                   int64_t table_stride, void* gx, void* gw, char* base, cudaStream_t s) {
    const int dt = h->c.dtype;
    LossFusedMaps maps{};
    cudaError_t e = launch_rows(h, L, rows, base, s);
    if (e != cudaSuccess) return cuda_fail(e);
    p.rows = at<float>(base, L.rows);
    p.unit = at<float>(base, L.unit);
    p.cols4 = L.cols4;
    if (!encode(&maps.x, dt, base + L.x, p.D, p.N, L.planes, L.pitch, 64)) return TBE_ERR_CUDA;
    Table w{h, table, table_stride, p.V, L.span, L.planes, L.pitch, direct(h, table, table_stride, p.V), base + L.w, L.w_bytes};
    const int64_t whole = w.is_direct ? p.V : std::min(p.V, L.span);
    const int walked = loss_fused_walk(p.D, L.planes);  // lines of a tile along the sum
    const int flush = loss_fused_flush(p.D, L.planes);
    p.x.tiles = (int)L.row_tiles;
    p.x.others = (int)((whole + walked - 1) / walked);
    p.x.part = at<float4>(base, L.x_part);
    p.x.out = gx;
    p.w.others = (int)((p.N + walked - 1) / walked);
    p.w.part = at<float4>(base, L.w_part);
    p.w.first = p.w.last = 1;
    p.w.tiles = (int)((whole + 127) / 128);
    {
        std::lock_guard<std::mutex> lock(h->choice_mu);
        auto& last = h->backward_choice;
        if (last.rows != p.N || last.items != whole) {
            choose_sides(&p.x, &p.w, p.D, h->num_sms);  // (of both, so that one alone has the same bits)
            last.x = p.x.slices;
            last.w = p.w.slices;
            last.rows = p.N;
            last.items = whole;
        }
        p.x.slices = last.x;
        p.w.slices = last.w;
    }
    if (!gx) p.x.tiles = 0;
    for (p.v0 = 0; p.v0 < p.V; p.v0 = p.v1) {
        p.v1 = std::min(p.V, p.v0 + whole);
        p.w0 = w.first(p.v0);
        e = w.fetch(p.v0, s);
        if (e != cudaSuccess) return cuda_fail(e);
        if (!w.map(&maps.w, p.v0)) return TBE_ERR_CUDA;
        p.x.others = (int)((p.v1 - p.v0 + walked - 1) / walked);
        p.x.first = p.v0 == 0;
        p.x.last = p.v1 == p.V;
        // (fp32's results take the parts of a sum as they come, 16-bit ones a whole sum)
        p.x.direct = p.x.slices == 1 && (L.planes == 3 || (p.x.first && p.x.last && p.x.others <= flush));
        p.w.direct = p.w.slices == 1 && (L.planes == 3 || p.w.others <= flush);
        p.w.tiles = gw ? (int)((p.v1 - p.v0 + 127) / 128) : 0;
        p.w.out = gw ? static_cast<char*>(gw) + p.v0 * p.D * elem_bytes(dt) : nullptr;
        e = launch_loss_fused(p, maps, dt, s);
        if (e != cudaSuccess) return cuda_fail(e);
        LossFinish f{p.x, p.w, p.N, p.v1 - p.v0, p.rows, p.unit, p.D, L.cols4};
        if (!p.x.last || p.x.direct) f.x.tiles = 0;
        if (p.w.direct) f.w.tiles = 0;
        if (f.x.tiles + f.w.tiles > 0) e = launch_loss_finish(f, dt, s);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return TBE_OK;
}

// Shares d's work items among the CTAs so that each ends at about the same
// time: the products are given out in turn, whose items are long, and d's fill
// up.  In blocks of 64 along the sum; an item of d is bound by its arithmetic, as
// long as ten of them, where it has fewer.
void share_d(LossStep* q, int ctas) {
    const int64_t x_cost = ((q->p_items + 63) / 64 + q->x_slabs - 1) / q->x_slabs;
    const int64_t w_cost = ((q->N + 63) / 64 + q->w_slabs - 1) / q->w_slabs;
    const int64_t d_cost = std::max((q->D + 63) / 64, 10);
    auto given = [&](int64_t items, int c) { return items / ctas + (c < items % ctas ? 1 : 0); };
    auto long_cost = [&](int c) {
        const int64_t w = given(q->n_gw, c);
        return w * w_cost + (given((int64_t)q->n_gw + q->n_gx, c) - w) * x_cost;
    };
    // the least level at which d's items find room, by halving
    int64_t lo = 0, hi = (int64_t)q->n_d * d_cost + 1;
    for (int c = 0; c < ctas; ++c) hi = std::max(hi, long_cost(c) + (int64_t)q->n_d * d_cost + 1);
    auto room = [&](int64_t level) {
        int64_t items = 0;
        for (int c = 0; c < ctas; ++c) items += std::max<int64_t>(0, level - long_cost(c)) / d_cost;
        return items;
    };
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (room(mid) >= q->n_d)
            hi = mid;
        else
            lo = mid + 1;
    }
    int64_t at = 0;
    for (int c = 0; c < ctas; ++c) {
        q->d_from[c] = (int32_t)at;
        at = std::min<int64_t>(q->n_d, at + std::max<int64_t>(0, lo - long_cost(c)) / d_cost);
    }
    q->d_from[ctas] = q->n_d;
}

int backward(const tbe_softmax_loss* h, const Plan& L, LossStep p, const RowsIn& rows, const void* table, int64_t table_stride,
             char* base, cudaStream_t s) {
    LossMaps maps{};
    const int dt = h->c.dtype;
    cudaError_t e = launch_rows(h, L, rows, base, s);
    if (e != cudaSuccess) return cuda_fail(e);
    p.rows = at<float>(base, L.rows);
    p.unit = at<float>(base, L.unit);
    p.row_tiles = (int)L.row_tiles;
    p.col_tiles = L.col_tiles;
    p.cols4 = L.cols4;
    p.x_part = at<float4>(base, L.x_part);
    if (!encode(&maps.x, dt, base + L.x, p.D, p.N, L.planes, L.pitch, 64)) return TBE_ERR_CUDA;
    Table w{h, table, table_stride, p.V, L.span, L.planes, L.pitch, direct(h, table, table_stride, p.V), base + L.w,
            L.w_bytes};

    // How the products' sums are cut: into items of about a quarter of a CTA's
    // share of a launch, so that none is waited for at its end.
    const int64_t piece = std::min(L.piece, p.V), item_tiles = (piece + 127) / 128;
    const int64_t row_blocks = (p.N + 63) / 64, piece_blocks = (piece + 63) / 64;
    const int64_t products = L.row_tiles * L.col_tiles * piece_blocks + item_tiles * L.col_tiles * row_blocks;
    const int64_t share = std::clamp<int64_t>(products / (h->num_sms * 2), 4, kLongSum / 64);
    auto slabs = [&](int64_t blocks, int64_t tiles) {
        const int64_t most = std::max<int64_t>(1, kMostParts / std::max<int64_t>(tiles, 1));
        return (int)std::min({most, blocks, (blocks + share - 1) / share});
    };
    p.x_slabs = slabs(piece_blocks, L.row_tiles * L.col_tiles);
    p.w_slabs = slabs(row_blocks, item_tiles * L.col_tiles);
    const int64_t pieces = (p.V + L.piece - 1) / L.piece;
    const int most_ctas = std::min(h->num_sms, kMaxStepCtas);
    for (int64_t j = 0; j <= pieces + 1; ++j) {
        LossStep q = p;
        q.n_d = q.n_gx = q.n_gw = q.n_fin_w = q.n_fin_x = 0;
        if (j < pieces) {
            q.d0 = j * L.piece;
            const int64_t items = std::min(L.piece, p.V - q.d0);
            q.n_d = (int)((items + 255) / 256 * L.row_tiles);
            q.dw0 = w.first(q.d0);
            e = w.fetch(q.d0, s);
            if (e != cudaSuccess) return cuda_fail(e);
            if (!w.map(&maps.w, q.d0) ||
                !encode(&maps.d_out, dt, base + L.d + (j & 1) * L.d_bytes, L.piece, p.N, L.planes, L.piece, 32))
                return TBE_ERR_CUDA;
        }
        if (j >= 1 && j <= pieces) {
            q.p0 = (j - 1) * L.piece;
            q.p_items = (int)std::min(L.piece, p.V - q.p0);
            q.pw0 = w.first(q.p0);
            q.first = j == 1;
            q.n_gx = p.gx ? (int)(L.row_tiles * L.col_tiles * p.x_slabs) : 0;
            q.n_gw = p.gw ? (int)((q.p_items + 127) / 128 * L.col_tiles * p.w_slabs) : 0;
            q.w_part = at<float4>(base, L.w_part + ((j - 1) & 1) * L.w_part_bytes);
            if (!w.map(&maps.pw, q.p0) ||
                !encode(&maps.d_in, dt, base + L.d + ((j - 1) & 1) * L.d_bytes, L.piece, p.N, L.planes, L.piece, 64))
                return TBE_ERR_CUDA;
        }
        if (j >= 2 && p.gw && p.w_slabs > 1) {
            q.f0 = (j - 2) * L.piece;
            q.f_items = (int)std::min(L.piece, p.V - q.f0);
            q.f_part = at<float4>(base, L.w_part + ((j - 2) & 1) * L.w_part_bytes);
            q.n_fin_w = (q.f_items + 127) / 128 * ((p.D + 31) / 32);
        }
        if (j == pieces + 1 && p.gx) q.n_fin_x = (int)L.row_tiles * ((p.D + 31) / 32);
        const int64_t n = (int64_t)q.n_d + q.n_gx + q.n_gw + q.n_fin_w + q.n_fin_x;
        if (n == 0) continue;
        const int ctas = (int)std::min<int64_t>(n, most_ctas);
        share_d(&q, ctas);
        e = launch_loss_step(q, maps, dt, ctas, s);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return TBE_OK;
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
    if (e == cudaSuccess) e = loss_mma_configure();
    if (e == cudaSuccess) e = loss_fused_configure();
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
    const size_t one = std::max(make_plan(h, N, V, false, false).total, make_plan(h, N, V, false, true).total);
    if (!backward) return one;
    return std::max({one, make_plan(h, N, V, true, false).total, make_plan(h, N, V, true, true).total});
}

int tbe_softmax_loss_forward(tbe_softmax_loss* h, const void* x, int64_t x_stride, const void* table,
                             int64_t table_stride, const void* targets, int32_t index_dtype, int64_t N, int64_t V,
                             float* loss, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range("tbe_softmax_loss_forward");
    const int rc = check(h, x, x_stride, table, table_stride, targets, index_dtype, N, V);
    if (rc) return rc;
    if (!workspace || !aligned16(workspace) || (N > 0 && (!loss || !lse))) return TBE_ERR_INVALID_ARG;
    if (workspace_bytes < tbe_softmax_loss_workspace_bytes(h, N, V, 0)) return TBE_ERR_WORKSPACE_TOO_SMALL;
    const int64_t row_bytes = N * (int64_t)sizeof(float), target_bytes = N * (index_dtype == TBE_I64 ? 8 : 4);
    if (overlap(loss, row_bytes, lse, row_bytes) || overlap(loss, row_bytes, targets, target_bytes) ||
        overlap(lse, row_bytes, targets, target_bytes))
        return TBE_ERR_INVALID_ARG;
    if (N == 0) return TBE_OK;
    LossForward p{};
    p.N = N, p.V = V, p.D = h->c.dim, p.c2 = argument_scale(h);
    p.targets = targets, p.index64 = index_dtype == TBE_I64, p.error = h->error;
    char* base = reinterpret_cast<char*>(align_up(reinterpret_cast<uintptr_t>(workspace)));
    return forward(h, make_plan(h, N, V, false, !direct(h, table, table_stride, V)), p, x, x_stride, table, table_stride, loss, lse, base,
                   static_cast<cudaStream_t>(stream));
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
    // (x is copied before a gradient is written; the table is read where it is)
    const int64_t bytes = elem_bytes(h->c.dtype), x_bytes = N * h->c.dim * bytes, w_bytes = V * h->c.dim * bytes;
    const int64_t table_bytes = V > 0 ? ((V - 1) * table_stride + h->c.dim) * bytes : 0;
    if (overlap(grad_x, x_bytes, table, table_bytes) || overlap(grad_table, w_bytes, table, table_bytes) ||
        overlap(grad_x, x_bytes, grad_table, w_bytes))
        return TBE_ERR_INVALID_ARG;
    if (N == 0) {
        if (!grad_table || V == 0) return TBE_OK;
        return status(cudaMemsetAsync(grad_table, 0, (size_t)w_bytes, s));
    }
    if (!grad_x && !grad_table) return TBE_OK;
    const Plan L = make_plan(h, N, V, true, !direct(h, table, table_stride, V));
    RowsIn rows{};
    rows.x = make_copy(h, x, x_stride, N, L.pitch, nullptr);
    rows.targets = targets, rows.index64 = index_dtype == TBE_I64, rows.V = V;
    rows.lse = lse, rows.g = grad_loss, rows.scale = h->c.scale, rows.error = h->error;
    char* base = reinterpret_cast<char*>(align_up(reinterpret_cast<uintptr_t>(workspace)));
    if (takes_fused(h)) {
        LossFused p{};
        p.N = N, p.V = V, p.D = h->c.dim, p.c2 = argument_scale(h), p.error = h->error;
        return backward_fused(h, L, p, rows, table, table_stride, grad_x, grad_table, base, s);
    }
    LossStep p{};
    p.N = N, p.V = V, p.D = h->c.dim, p.c2 = argument_scale(h);
    p.gx = grad_x, p.gw = grad_table, p.error = h->error;
    return backward(h, L, p, rows, table, table_stride, base, s);
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
