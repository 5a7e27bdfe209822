// gradclip.cu -- the global gradient norm over many tensors, and clipping by
// it (cns_grad_norm, cns_grad_clip).
//
//   norm = sqrt(sum over all tensors of x^2)   (or the largest |x|)
//   out  = x * min(1, max_norm / (norm + eps))
//
// Tensors are cut into tiles of kTileBytes at 16-byte boundaries of the
// address space (so a tile's vectors are aligned wherever its tensor starts;
// only a tensor's first and last vector can be partial).  One warp takes one
// tile.  The table of tensors goes to the workspace as kernel arguments of
// small launches: no staging buffer, nothing for a graph capture to lose.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "cns.h"
#include "cns_host.h"
#include "step_device.cuh"

namespace cns {
namespace {

constexpr int kTileBytes = 4096;
constexpr int kTileVecs = kTileBytes / 16;      // 16-byte vectors of a tile
constexpr int kLaneVecs = kTileVecs / 32;       // of one lane

// One tensor of the table.
struct GradEntry {
    uint64_t src;
    uint64_t dst;
    int64_t elems;
    uint32_t tile0;   // the tensor's first tile among all tensors' tiles
    uint32_t types;   // dtype of src | dtype of dst << 8
};
static_assert(sizeof(GradEntry) == 32, "table entries are two 16-byte units");

constexpr int kChunkEntries = 120;
struct TableChunk {
    GradEntry e[kChunkEntries];
    GradEntry *to;
    int32_t n;
};

__global__ void grad_table_kernel(const __grid_constant__ TableChunk c)
{
    for (int i = threadIdx.x; i < c.n; i += blockDim.x)
        c.to[i] = c.e[i];
}

struct GradParams {
    const GradEntry *table;
    double *partial;       // one per CTA
    uint32_t *status;
    float *norm;
    float *factor;
    int32_t count;
    uint32_t tiles;
    float max_norm, eps;
};

// Largest i with table[i].tile0 <= tile (tensors without elements have no
// tiles and are not in the table).
__device__ __forceinline__ int find_tensor(const GradEntry *table, int count, uint32_t tile)
{
    int lo = 0, hi = count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (table[mid].tile0 <= tile)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// One 16-byte vector's elements as floats.
template <int D> struct Vec {
    static constexpr int N = 16 / static_cast<int>(sizeof(typename Elem<D>::type));
    static __device__ __forceinline__ void unpack(const uint4 &v, float *f)
    {
        const typename Elem<D>::type *e = reinterpret_cast<const typename Elem<D>::type *>(&v);
#pragma unroll
        for (int i = 0; i < N; ++i)
            f[i] = Elem<D>::get(e[i]);
    }
};

// Calls body(first element index in the tensor, count, values) for the
// calling lane's vectors of a tile.  Vectors that the tensor covers only in
// part are loaded element by element; body gets the elements that are there.
template <int D, class Body>
__device__ __forceinline__ void for_tile(const GradEntry &t, uint32_t tile, Body body)
{
    using T = typename Elem<D>::type;
    constexpr int N = Vec<D>::N;
    const uint64_t end = t.src + static_cast<uint64_t>(t.elems) * sizeof(T);
    const uint64_t base = (t.src & ~15ull) + static_cast<uint64_t>(tile - t.tile0) * kTileBytes;
    const uint32_t lane = threadIdx.x & 31u;
#pragma unroll
    for (int j = 0; j < kLaneVecs; ++j) {
        const uint64_t a = base + (static_cast<uint64_t>(j) * 32 + lane) * 16;
        if (a + 16 <= t.src || a >= end)
            continue;
        float f[N];
        if (a >= t.src && a + 16 <= end) {
            const uint4 v = *reinterpret_cast<const uint4 *>(a);
            Vec<D>::unpack(v, f);
            body(static_cast<int64_t>((a - t.src) / sizeof(T)), N, f);
        } else {
            const uint64_t from = a < t.src ? t.src : a, to = a + 16 < end ? a + 16 : end;
            const int n = static_cast<int>((to - from) / sizeof(T));
            for (int i = 0; i < n; ++i)
                f[0] = Elem<D>::get(reinterpret_cast<const T *>(from)[i]),
                body(static_cast<int64_t>((from - t.src) / sizeof(T)) + i, 1, f);
        }
    }
}

template <int NORM>
__device__ __forceinline__ void accumulate(float &acc, const float *f, int n)
{
    for (int i = 0; i < n; ++i) {
        if constexpr (NORM == CNS_NORM_L2)
            acc = fmaf(f[i], f[i], acc);
        else   // magnitudes compare as integers, NaN above inf
            acc = __uint_as_float(max(__float_as_uint(acc), __float_as_uint(fabsf(f[i]))));
    }
}

template <int NORM>
__global__ void __launch_bounds__(256) grad_partial_kernel(const GradParams p)
{
    const uint32_t warps = gridDim.x * (blockDim.x >> 5);
    double total = 0.0;
    float most = 0.f;
    for (uint32_t tile = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); tile < p.tiles; tile += warps) {
        const GradEntry t = p.table[find_tensor(p.table, p.count, tile)];
        float acc = 0.f;
        auto body = [&](int64_t, int n, const float *f) { accumulate<NORM>(acc, f, n); };
        switch (t.types & 0xffu) {
        case CNS_DT_F32: for_tile<CNS_DT_F32>(t, tile, body); break;
        case CNS_DT_BF16: for_tile<CNS_DT_BF16>(t, tile, body); break;
        default: for_tile<CNS_DT_F16>(t, tile, body); break;
        }
        if (NORM == CNS_NORM_L2)
            total += static_cast<double>(acc);
        else
            accumulate<NORM>(most, &acc, 1);
    }
    __shared__ double s_sum[8];
    __shared__ float s_most[8];
    if (NORM == CNS_NORM_L2) {
        total = warp_sum(total);
    } else {
        most = __uint_as_float(__reduce_max_sync(kFullWarp, __float_as_uint(most)));
    }
    if ((threadIdx.x & 31u) == 0) {
        s_sum[threadIdx.x >> 5] = total;
        s_most[threadIdx.x >> 5] = most;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (uint32_t w = 1; w < (blockDim.x >> 5); ++w) {
            total += s_sum[w];
            accumulate<NORM>(most, &s_most[w], 1);
        }
        p.partial[blockIdx.x] = NORM == CNS_NORM_L2 ? total : static_cast<double>(most);
    }
}

template <int NORM>
__global__ void __launch_bounds__(32) grad_join_kernel(const GradParams p, int n)
{
    double total = 0.0;
    float most = 0.f;
    for (int i = threadIdx.x; i < n; i += 32) {
        total += p.partial[i];
        const float f = static_cast<float>(p.partial[i]);
        accumulate<NORM>(most, &f, 1);
    }
    if (NORM == CNS_NORM_L2)
        total = warp_sum(total);
    else
        most = __uint_as_float(__reduce_max_sync(kFullWarp, __float_as_uint(most)));
    if (threadIdx.x == 0) {
        const float norm = NORM == CNS_NORM_L2 ? static_cast<float>(sqrt(total)) : most;
        *p.norm = norm;
        const float f = p.max_norm / (norm + p.eps);
        *p.factor = f < 1.f || f != f ? f : 1.f;
    }
}

template <int D>
__device__ __forceinline__ void store(uint64_t dst, int64_t at, const float *f, int n)
{
    typename Elem<D>::type *o = reinterpret_cast<typename Elem<D>::type *>(dst) + at;
    for (int i = 0; i < n; ++i)
        o[i] = Elem<D>::put(f[i]);
}

__global__ void __launch_bounds__(256) grad_scale_kernel(const GradParams p)
{
    const uint32_t warps = gridDim.x * (blockDim.x >> 5);
    const float factor = *p.factor;
    for (uint32_t tile = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); tile < p.tiles; tile += warps) {
        const GradEntry t = p.table[find_tensor(p.table, p.count, tile)];
        auto body = [&](int64_t at, int n, float *f) {
            for (int i = 0; i < n; ++i)
                f[i] *= factor;
            switch (t.types >> 8) {
            case CNS_DT_F32: store<CNS_DT_F32>(t.dst, at, f, n); break;
            case CNS_DT_BF16: store<CNS_DT_BF16>(t.dst, at, f, n); break;
            default: store<CNS_DT_F16>(t.dst, at, f, n); break;
            }
        };
        switch (t.types & 0xffu) {
        case CNS_DT_F32: for_tile<CNS_DT_F32>(t, tile, body); break;
        case CNS_DT_BF16: for_tile<CNS_DT_BF16>(t, tile, body); break;
        default: for_tile<CNS_DT_F16>(t, tile, body); break;
        }
    }
}

constexpr int kMaxPartials = 1024;

size_t workspace_bytes(int64_t count)
{
    return CNS_STEP_WORKSPACE_HEADER_BYTES + kMaxPartials * sizeof(double) + 128 +
           static_cast<size_t>(count) * sizeof(GradEntry);
}

int64_t elem_bytes(int32_t dtype) { return dtype == CNS_DT_F32 ? 4 : 2; }

int check_tensor(const cns_tensor_t &t)
{
    if (t.elems < 0 || t.elems > (1ll << 42) || t.dtype < CNS_DT_F32 || t.dtype > CNS_DT_F16 || t.reserved != 0)
        return CNS_ERR_INVALID_VALUE;
    if (t.elems == 0)
        return CNS_SUCCESS;
    if (!t.data_dev)
        return CNS_ERR_NULL_PTR;
    return reinterpret_cast<uintptr_t>(t.data_dev) % elem_bytes(t.dtype) ? CNS_ERR_INVALID_VALUE : CNS_SUCCESS;
}

int64_t tiles_of(const cns_tensor_t &t)
{
    const uint64_t a = reinterpret_cast<uint64_t>(t.data_dev);
    return static_cast<int64_t>(((a & 15u) + t.elems * elem_bytes(t.dtype) + kTileBytes - 1) / kTileBytes);
}

template <bool CLIP>
int grad_run(cns_grad_clip_t *g)
{
    if (!g)
        return CNS_ERR_NULL_PTR;
    if (g->count < 0 || g->count > CNS_GRAD_MAX_TENSORS || g->norm_type < CNS_NORM_L2 || g->norm_type > CNS_NORM_INF)
        return CNS_ERR_INVALID_VALUE;
    if (CLIP && (!(g->max_norm >= 0.f) || !(g->eps >= 0.f) || !std::isfinite(g->eps)))
        return CNS_ERR_INVALID_VALUE;
    if (!g->norm_dev || !g->workspace_dev || (g->count > 0 && !g->grads))
        return CNS_ERR_NULL_PTR;
    if (reinterpret_cast<uintptr_t>(g->norm_dev) % 4 ||
        reinterpret_cast<uintptr_t>(g->workspace_dev) % CNS_STEP_WORKSPACE_ALIGN ||
        g->workspace_bytes < workspace_bytes(g->count))
        return CNS_ERR_INVALID_VALUE;
    int64_t tiles = 0;
    for (int64_t i = 0; i < g->count; ++i) {
        if (int rc = check_tensor(g->grads[i]))
            return rc;
        if (CLIP && g->outs) {
            if (int rc = check_tensor(g->outs[i]))
                return rc;
            if (g->outs[i].elems != g->grads[i].elems)
                return CNS_ERR_INVALID_VALUE;
            if (g->outs[i].data_dev == g->grads[i].data_dev && g->outs[i].dtype != g->grads[i].dtype &&
                g->grads[i].elems > 0)
                return CNS_ERR_INVALID_VALUE;
        }
        if (g->grads[i].elems)
            tiles += tiles_of(g->grads[i]);
    }
    if (tiles > 0x7fffffff)
        return CNS_ERR_INVALID_VALUE;
    DeviceInfo dev;
    if (int rc = current_device(&dev))
        return rc;
    cudaStream_t s = to_stream(g->stream);
    char *ws = static_cast<char *>(g->workspace_dev);
    GradParams p = {};
    p.partial = reinterpret_cast<double *>(ws + CNS_STEP_WORKSPACE_HEADER_BYTES);
    p.factor = reinterpret_cast<float *>(p.partial + kMaxPartials);
    GradEntry *table = reinterpret_cast<GradEntry *>(ws + CNS_STEP_WORKSPACE_HEADER_BYTES +
                                                     kMaxPartials * sizeof(double) + 128);
    p.table = table;
    p.status = reinterpret_cast<uint32_t *>(ws) + kStepStatusWord;
    p.norm = g->norm_dev;
    p.tiles = static_cast<uint32_t>(tiles);
    p.max_norm = g->max_norm;
    p.eps = g->eps;
    TableChunk c;
    c.n = 0;
    uint32_t tile0 = 0;
    for (int64_t i = 0; i < g->count; ++i) {
        const cns_tensor_t &t = g->grads[i];
        if (t.elems) {
            const cns_tensor_t &o = CLIP && g->outs ? g->outs[i] : t;
            c.e[c.n++] = GradEntry{reinterpret_cast<uint64_t>(t.data_dev), reinterpret_cast<uint64_t>(o.data_dev),
                                   t.elems, tile0, static_cast<uint32_t>(t.dtype | o.dtype << 8)};
            tile0 += static_cast<uint32_t>(tiles_of(t));
        }
        if (c.n == kChunkEntries || (c.n > 0 && i + 1 == g->count)) {
            c.to = table + p.count;
            grad_table_kernel<<<1, 128, 0, s>>>(c);
            p.count += c.n;
            c.n = 0;
        }
    }
    const int ctas = static_cast<int>(std::min<int64_t>((tiles + 7) / 8, std::min(kMaxPartials, dev.sm_count * 6)));
    const bool l2 = g->norm_type == CNS_NORM_L2;
    if (ctas > 0) {
        if (l2)
            grad_partial_kernel<CNS_NORM_L2><<<ctas, 256, 0, s>>>(p);
        else
            grad_partial_kernel<CNS_NORM_INF><<<ctas, 256, 0, s>>>(p);
    }
    if (l2)
        grad_join_kernel<CNS_NORM_L2><<<1, 32, 0, s>>>(p, ctas);
    else
        grad_join_kernel<CNS_NORM_INF><<<1, 32, 0, s>>>(p, ctas);
    if (CLIP && ctas > 0)
        grad_scale_kernel<<<ctas, 256, 0, s>>>(p);
    CNS_CUDA(cudaGetLastError());
    if (!g->sync)
        return CNS_SUCCESS;
    g->device_status = 0;
    return syncall_read_workspace(g->workspace_dev, g->stream, nullptr, nullptr, &g->device_status);
}

}  // namespace
}  // namespace cns

using namespace cns;

extern "C" int cns_grad_workspace_bytes(int64_t count, size_t *bytes)
{
    if (!bytes)
        return CNS_ERR_NULL_PTR;
    if (count < 0 || count > CNS_GRAD_MAX_TENSORS)
        return CNS_ERR_INVALID_VALUE;
    *bytes = workspace_bytes(count);
    return CNS_SUCCESS;
}

extern "C" int cns_grad_norm(cns_grad_clip_t *g)
{
    TraceRange tr("cns_grad_norm", g ? static_cast<uint64_t>(g->count) : 0);
    return grad_run<false>(g);
}

extern "C" int cns_grad_clip(cns_grad_clip_t *g)
{
    TraceRange tr("cns_grad_clip", g ? static_cast<uint64_t>(g->count) : 0);
    return grad_run<true>(g);
}

extern "C" int cns_step_workspace_init(void *ws_dev, size_t bytes, cns_stream_t stream)
{
    if (!ws_dev)
        return CNS_ERR_NULL_PTR;
    if (bytes < CNS_STEP_WORKSPACE_HEADER_BYTES || reinterpret_cast<uintptr_t>(ws_dev) % CNS_STEP_WORKSPACE_ALIGN)
        return CNS_ERR_INVALID_VALUE;
    DeviceInfo dev;
    if (int rc = current_device(&dev))
        return rc;
    CNS_CUDA(cudaMemsetAsync(ws_dev, 0, CNS_STEP_WORKSPACE_HEADER_BYTES, to_stream(stream)));
    return CNS_SUCCESS;
}
