// expert_rows.cu -- rows to their experts and back (cns_dispatch, cns_combine,
// cns_combine_backward).
//
//   dispatch           rows[places[t][j]] = x[t]
//   combine            y[t] = base[t] + sum_j w[t][j] rows[places[t][j]]
//   combine's gradient drows[places[t][j]] = w[t][j] dy[t],
//                      dw[t][j] = sum over the columns of dy[t] rows[places[t][j]]
//
// All go by tokens, not by rows: what a token has is read or written once and
// its top_k rows once each, wherever they are, so the traffic is the operands'
// own bytes and no sum needs an atomic.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "cns.h"
#include "cns_host.h"
#include "rows_device.cuh"

namespace cns {
namespace {

// How a CTA's threads lie over tokens and a row's accesses: `per` whole tokens of `units` accesses each, or
// (per = 1) one of `parts` stretches of `span` accesses of a token.
struct Tiling {
    uint32_t units, per, parts, span, threads, ctas;
};

constexpr uint32_t kRowThreads = 256;

bool tile(int64_t tokens, int64_t units, Tiling *t)
{
    t->units = static_cast<uint32_t>(units);
    t->per = std::max<uint32_t>(1u, kRowThreads / t->units);
    t->parts = (t->units + kRowThreads - 1) / kRowThreads;
    t->span = (t->units + t->parts - 1) / t->parts;
    t->threads = (t->per * t->span + 31) / 32 * 32;
    const int64_t ctas = (tokens + t->per - 1) / t->per * t->parts;
    t->ctas = static_cast<uint32_t>(ctas);
    return ctas <= 0x7fffffff;
}

// The calling thread's token and access; false if it has none.
__device__ __forceinline__ bool my_place(const Tiling &m, uint32_t cta, int64_t tokens, int64_t *t, uint32_t *u)
{
    if (m.parts == 1) {
        const uint32_t k = threadIdx.x / m.units;
        *t = static_cast<int64_t>(cta) * m.per + k;
        *u = threadIdx.x - k * m.units;
        return k < m.per && *t < tokens;
    }
    *t = cta / m.parts;
    *u = cta % m.parts * m.span + threadIdx.x;
    return threadIdx.x < m.span && *u < m.units;
}

struct DispatchParams {
    const uint8_t *x;
    uint8_t *rows;
    const uint8_t *scales;
    uint8_t *row_scales;
    const int32_t *places;
    int64_t tokens, x_stride, rows_stride, scales_stride, row_scales_stride;
    uint32_t limit;   // rows
    int32_t top_k, scale_access;
    Tiling data, scale;
};

template <int A>
__device__ __forceinline__ void move(const DispatchParams &p, const Tiling &m, uint32_t cta, const uint8_t *from,
                                     int64_t from_stride, uint8_t *to, int64_t to_stride)
{
    using B = typename Bits<A>::type;
    int64_t t;
    uint32_t u;
    if (!my_place(m, cta, p.tokens, &t, &u))
        return;
    const B v = *reinterpret_cast<const B *>(from + t * from_stride + static_cast<int64_t>(u) * A);
    const int32_t *place = p.places + t * p.top_k;
    to += static_cast<int64_t>(u) * A;
#pragma unroll 4
    for (int j = 0; j < p.top_k; ++j) {
        const uint32_t row = static_cast<uint32_t>(place[j]);
        if (row < p.limit)
            *reinterpret_cast<B *>(to + row * to_stride) = v;
    }
}

template <int A>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(const __grid_constant__ DispatchParams p)
{
    grid_dependency_wait();
    if (blockIdx.x < p.data.ctas) {
        move<A>(p, p.data, blockIdx.x, p.x, p.x_stride, p.rows, p.rows_stride);
        return;
    }
    const uint32_t cta = blockIdx.x - p.data.ctas;
    if (p.scale_access == 16)
        move<16>(p, p.scale, cta, p.scales, p.scales_stride, p.row_scales, p.row_scales_stride);
    else if (p.scale_access == 4)
        move<4>(p, p.scale, cta, p.scales, p.scales_stride, p.row_scales, p.row_scales_stride);
    else
        move<1>(p, p.scale, cta, p.scales, p.scales_stride, p.row_scales, p.row_scales_stride);
}

struct CombineParams {
    const void *rows;
    const int32_t *places;
    const float *weights;
    const void *base;
    void *y;
    int64_t tokens, rows_stride, base_stride, y_stride;   // elements
    uint32_t limit;
    int32_t top_k;
    Tiling data;
};

constexpr int kBatch = 4;   // rows in flight a thread

template <int D, int A>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const __grid_constant__ CombineParams p)
{
    using T = typename Elem<D>::type;
    using B = typename Bits<A>::type;
    constexpr int V = A / static_cast<int>(sizeof(T));
    grid_dependency_wait();
    int64_t t;
    uint32_t u;
    if (!my_place(p.data, blockIdx.x, p.tokens, &t, &u))
        return;
    const T *rows = static_cast<const T *>(p.rows) + static_cast<int64_t>(u) * V;
    const int32_t *place = p.places + t * p.top_k;
    const float *weight = p.weights + t * p.top_k;
    float sum[V] = {};
    for (int j = 0; j < p.top_k; j += kBatch) {
        B raw[kBatch];
        float w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const uint32_t row = j + i < p.top_k ? static_cast<uint32_t>(place[j + i]) : 0xffffffffu;
            raw[i] = B{};
            w[i] = 0.f;
            if (row < p.limit) {
                raw[i] = *reinterpret_cast<const B *>(rows + row * p.rows_stride);
                w[i] = p.weights ? weight[j + i] : 1.f;
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float v[V];
            unpack<D, A>(raw[i], v);
#pragma unroll
            for (int k = 0; k < V; ++k)
                sum[k] = fmaf(w[i], v[k], sum[k]);
        }
    }
    if (p.base) {
        float v[V];
        unpack<D, A>(*reinterpret_cast<const B *>(static_cast<const T *>(p.base) + t * p.base_stride + static_cast<int64_t>(u) * V), v);
#pragma unroll
        for (int k = 0; k < V; ++k)
            sum[k] += v[k];
    }
    *reinterpret_cast<B *>(static_cast<T *>(p.y) + t * p.y_stride + static_cast<int64_t>(u) * V) = pack<D, A>(sum);
}

struct CombineGradParams {
    const void *rows;
    const void *dy;
    const int32_t *places;
    const float *weights;
    void *drows;
    float *dweights;
    int64_t tokens, rows_stride, dy_stride, drows_stride;   // elements
    uint32_t limit, units;
    int32_t top_k;
};

constexpr int kGradUnits = 2;   // accesses of a row that a thread holds

// LANES threads take a token: of a warp (8 or 32), or the CTA (0).
template <int D, int A, int LANES>
__global__ void __launch_bounds__(kRowThreads) combine_backward_kernel(const __grid_constant__ CombineGradParams p)
{
    using T = typename Elem<D>::type;
    using B = typename Bits<A>::type;
    constexpr int V = A / static_cast<int>(sizeof(T));
    constexpr int kLanes = LANES ? LANES : 32;   // that sum by shuffles
    __shared__ float s_dot[kRowThreads / kLanes][CNS_ROUTE_MAX_TOP_K];
    const uint32_t lanes = LANES ? LANES : blockDim.x;
    const uint32_t g = LANES ? threadIdx.x % lanes : threadIdx.x, slot = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
    const int64_t t = LANES ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes : blockIdx.x;
    const bool token = t < p.tokens;
    grid_dependency_wait();
    for (int j = l; j < p.top_k; j += kLanes)
        s_dot[slot][j] = 0.f;
    __syncwarp();
    const int32_t *place = p.places + t * p.top_k;
    const float *weight = p.weights + t * p.top_k;
    for (uint32_t u0 = 0; u0 < p.units; u0 += lanes * kGradUnits) {
        float dy[kGradUnits][V];
        bool mine[kGradUnits];
#pragma unroll
        for (int k = 0; k < kGradUnits; ++k) {
            const uint32_t u = u0 + k * lanes + g;
            mine[k] = token && u < p.units;
            B raw = B{};
            if (mine[k])
                raw = *reinterpret_cast<const B *>(static_cast<const T *>(p.dy) + t * p.dy_stride + static_cast<int64_t>(u) * V);
            unpack<D, A>(raw, dy[k]);
        }
        for (int j = 0; j < p.top_k; j += 2) {
            uint32_t row[2];
            B raw[2][kGradUnits];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                row[i] = token && j + i < p.top_k ? static_cast<uint32_t>(place[j + i]) : 0xffffffffu;
#pragma unroll
                for (int k = 0; k < kGradUnits; ++k) {
                    raw[i][k] = B{};
                    if (p.dweights && mine[k] && row[i] < p.limit)
                        raw[i][k] = *reinterpret_cast<const B *>(static_cast<const T *>(p.rows) + row[i] * p.rows_stride +
                                                                 static_cast<int64_t>(u0 + k * lanes + g) * V);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool there = row[i] < p.limit;
                if (p.drows && there) {
                    const float w = p.weights ? weight[j + i] : 1.f;
#pragma unroll
                    for (int k = 0; k < kGradUnits; ++k) {
                        float v[V];
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            v[e] = w * dy[k][e];
                        if (mine[k])
                            *reinterpret_cast<B *>(static_cast<T *>(p.drows) + row[i] * p.drows_stride +
                                                   static_cast<int64_t>(u0 + k * lanes + g) * V) = pack<D, A>(v);
                    }
                }
                if (p.dweights && j + i < p.top_k) {
                    float dot = 0.f;
                    if (there) {
#pragma unroll
                        for (int k = 0; k < kGradUnits; ++k) {
                            float v[V];
                            unpack<D, A>(raw[i][k], v);
#pragma unroll
                            for (int e = 0; e < V; ++e)
                                dot = fmaf(dy[k][e], v[e], dot);
                        }
                    }
#pragma unroll
                    for (int d = kLanes / 2; d > 0; d >>= 1)
                        dot += __shfl_xor_sync(kFullWarp, dot, d);
                    if (l == 0)
                        s_dot[slot][j + i] += dot;
                }
            }
        }
    }
    if (!p.dweights)
        return;
    if (LANES)
        __syncwarp();
    else
        __syncthreads();
    if (!token)
        return;
    for (int j = g; j < p.top_k; j += lanes) {
        float dot = s_dot[slot][j];
        if (!LANES) {
            dot = 0.f;
            for (uint32_t i = 0; i < blockDim.x / 32; ++i)
                dot += s_dot[i][j];
        }
        p.dweights[t * p.top_k + j] = dot;
    }
}

template <class P>
cudaError_t launch(void (*kernel)(P), const P &p, uint32_t ctas, uint32_t threads, cudaStream_t s)
{
    cudaLaunchAttribute early;
    cudaLaunchConfig_t cfg = early_launch(&early);
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D>
cudaError_t launch_combine(const CombineParams &p, int access, cudaStream_t s)
{
    constexpr int E = sizeof(typename Elem<D>::type);
    return launch(access == 16  ? combine_kernel<D, 16>
                  : access == 8 ? combine_kernel<D, 8>
                  : access == 4 ? combine_kernel<D, 4>
                                : combine_kernel<D, E>,
                  p, p.data.ctas, p.data.threads, s);
}

template <int D, int A>
cudaError_t launch_grad(const CombineGradParams &p, cudaStream_t s)
{
    // a token's lanes: enough for the row's accesses, so that few idle and few sums meet in shared memory
    if (p.units <= 8 * kGradUnits)
        return launch(combine_backward_kernel<D, A, 8>, p, static_cast<uint32_t>((p.tokens + 31) / 32), kRowThreads, s);
    if (p.units <= 32 * kGradUnits)
        return launch(combine_backward_kernel<D, A, 32>, p, static_cast<uint32_t>((p.tokens + 7) / 8), kRowThreads, s);
    const uint32_t threads = std::min(kRowThreads, (p.units + 32 * kGradUnits - 1) / (32 * kGradUnits) * 32);
    return launch(combine_backward_kernel<D, A, 0>, p, static_cast<uint32_t>(p.tokens), threads, s);
}

template <int D>
cudaError_t launch_combine_backward(const CombineGradParams &p, int access, cudaStream_t s)
{
    constexpr int E = sizeof(typename Elem<D>::type);
    return access == 16  ? launch_grad<D, 16>(p, s)
           : access == 8 ? launch_grad<D, 8>(p, s)
           : access == 4 ? launch_grad<D, 4>(p, s)
                         : launch_grad<D, E>(p, s);
}

bool sizes_ok(int64_t tokens, int64_t rows, int32_t top_k, int32_t reserved)
{
    return tokens >= 0 && rows >= 0 && top_k >= 1 && top_k <= CNS_ROUTE_MAX_TOP_K && tokens <= 0x7fffffff / top_k &&
           reserved == 0;
}

// A matrix's stride in elements (`packed` where it is 0); false if it is too small or not to be counted in bytes.
bool stride_ok(int64_t given, int64_t packed, int64_t *stride)
{
    *stride = given ? given : packed;
    return *stride >= packed && *stride <= (INT64_MAX >> 34);
}

bool off(const void *p, int64_t bytes) { return address(p) % bytes != 0; }

uint32_t row_limit(int64_t rows) { return static_cast<uint32_t>(std::min<int64_t>(rows, 0x80000000ll)); }

}  // namespace
}  // namespace cns

using namespace cns;

extern "C" int cns_dispatch(const cns_dispatch_t *d)
{
    TraceRange tr("cns_dispatch", d ? static_cast<uint64_t>(d->tokens) : 0);
    if (!d)
        return CNS_ERR_NULL_PTR;
    const bool scales = d->scales_dev != nullptr;
    DispatchParams p = {};
    if (!sizes_ok(d->tokens, d->rows, d->top_k, d->reserved) || d->row_bytes < 1 || d->row_bytes > CNS_ROWS_MAX_BYTES ||
        !stride_ok(d->x_stride, d->row_bytes, &p.x_stride) || !stride_ok(d->rows_stride, d->row_bytes, &p.rows_stride))
        return CNS_ERR_INVALID_VALUE;
    if (!scales && (d->row_scales_dev || d->scale_bytes))
        return CNS_ERR_INVALID_VALUE;
    if (scales && (d->scale_bytes < 1 || d->scale_bytes > CNS_ROWS_MAX_BYTES ||
                   !stride_ok(d->scales_stride, d->scale_bytes, &p.scales_stride) ||
                   !stride_ok(d->row_scales_stride, d->scale_bytes, &p.row_scales_stride)))
        return CNS_ERR_INVALID_VALUE;
    if (d->tokens > 0 && (!d->x_dev || !d->places_dev || (d->rows > 0 && (!d->rows_dev || (scales && !d->row_scales_dev)))))
        return CNS_ERR_NULL_PTR;
    if (off(d->places_dev, 4) || (d->rows_dev && d->rows_dev == d->x_dev) || (scales && d->row_scales_dev == d->scales_dev))
        return CNS_ERR_INVALID_VALUE;
    p.x = static_cast<const uint8_t *>(d->x_dev);
    p.rows = static_cast<uint8_t *>(d->rows_dev);
    p.scales = static_cast<const uint8_t *>(d->scales_dev);
    p.row_scales = static_cast<uint8_t *>(d->row_scales_dev);
    p.places = d->places_dev;
    p.tokens = d->tokens;
    p.limit = row_limit(d->rows);
    p.top_k = d->top_k;
    const int access = access_bytes(address(p.x) | address(p.rows) | d->row_bytes | p.x_stride | p.rows_stride);
    if (!tile(p.tokens, d->row_bytes / access, &p.data))
        return CNS_ERR_INVALID_VALUE;
    if (scales) {
        const int a = access_bytes(address(p.scales) | address(p.row_scales) | d->scale_bytes | p.scales_stride | p.row_scales_stride);
        p.scale_access = a == 16 ? 16 : a >= 4 ? 4 : 1;
        if (!tile(p.tokens, d->scale_bytes / p.scale_access, &p.scale))
            return CNS_ERR_INVALID_VALUE;
    }
    const int64_t ctas = static_cast<int64_t>(p.data.ctas) + p.scale.ctas;
    if (ctas > 0x7fffffff)
        return CNS_ERR_INVALID_VALUE;
    DeviceInfo dev;
    if (int rc = current_device(&dev))
        return rc;
    if (p.tokens == 0 || d->rows == 0)
        return CNS_SUCCESS;
    const uint32_t threads = std::max(p.data.threads, p.scale.threads);
    CNS_CUDA(launch(access == 16  ? dispatch_kernel<16>
                    : access == 8 ? dispatch_kernel<8>
                    : access == 4 ? dispatch_kernel<4>
                    : access == 2 ? dispatch_kernel<2>
                                  : dispatch_kernel<1>,
                    p, static_cast<uint32_t>(ctas), threads, to_stream(d->stream)));
    return CNS_SUCCESS;
}

extern "C" int cns_combine(const cns_combine_t *c)
{
    TraceRange tr("cns_combine", c ? static_cast<uint64_t>(c->tokens) : 0);
    if (!c)
        return CNS_ERR_NULL_PTR;
    CombineParams p = {};
    if (!sizes_ok(c->tokens, c->rows, c->top_k, c->reserved) || c->width < 1 || c->width > CNS_ROWS_MAX_BYTES / 4 ||
        c->dtype < CNS_DT_F32 || c->dtype > CNS_DT_F16 || !stride_ok(c->rows_stride, c->width, &p.rows_stride) ||
        !stride_ok(c->base_stride, c->width, &p.base_stride) || !stride_ok(c->y_stride, c->width, &p.y_stride))
        return CNS_ERR_INVALID_VALUE;
    if (c->tokens > 0 && (!c->places_dev || !c->y_dev || (c->rows > 0 && !c->rows_dev)))
        return CNS_ERR_NULL_PTR;
    const int64_t e = c->dtype == CNS_DT_F32 ? 4 : 2;
    if (off(c->rows_dev, e) || off(c->base_dev, e) || off(c->y_dev, e) || off(c->places_dev, 4) || off(c->weights_dev, 4) ||
        (c->y_dev && (c->y_dev == c->rows_dev || (c->y_dev == c->base_dev && p.y_stride != p.base_stride))))
        return CNS_ERR_INVALID_VALUE;
    p.rows = c->rows_dev;
    p.places = c->places_dev;
    p.weights = c->weights_dev;
    p.base = c->base_dev;
    p.y = c->y_dev;
    p.tokens = c->tokens;
    p.limit = row_limit(c->rows);
    p.top_k = c->top_k;
    uint64_t bits = address(p.rows) | address(p.y) | (c->width * e) | (p.rows_stride * e) | (p.y_stride * e);
    if (p.base)
        bits |= address(p.base) | (p.base_stride * e);
    const int access = access_bytes(bits);
    if (!tile(p.tokens, c->width * e / access, &p.data))
        return CNS_ERR_INVALID_VALUE;
    DeviceInfo dev;
    if (int rc = current_device(&dev))
        return rc;
    if (p.tokens == 0)
        return CNS_SUCCESS;
    cudaStream_t s = to_stream(c->stream);
    CNS_CUDA(c->dtype == CNS_DT_F32    ? launch_combine<CNS_DT_F32>(p, access, s)
             : c->dtype == CNS_DT_BF16 ? launch_combine<CNS_DT_BF16>(p, access, s)
                                       : launch_combine<CNS_DT_F16>(p, access, s));
    return CNS_SUCCESS;
}

extern "C" int cns_combine_backward(const cns_combine_grad_t *g)
{
    TraceRange tr("cns_combine_backward", g ? static_cast<uint64_t>(g->tokens) : 0);
    if (!g)
        return CNS_ERR_NULL_PTR;
    CombineGradParams p = {};
    if (!sizes_ok(g->tokens, g->rows, g->top_k, g->reserved) || g->width < 1 || g->width > CNS_ROWS_MAX_BYTES / 4 ||
        g->dtype < CNS_DT_F32 || g->dtype > CNS_DT_F16 || !stride_ok(g->rows_stride, g->width, &p.rows_stride) ||
        !stride_ok(g->dy_stride, g->width, &p.dy_stride) || !stride_ok(g->drows_stride, g->width, &p.drows_stride))
        return CNS_ERR_INVALID_VALUE;
    if (g->tokens > 0 && (!g->places_dev || !g->dy_dev || (!g->drows_dev && !g->dweights_dev) ||
                          (g->rows > 0 && g->dweights_dev && !g->rows_dev)))
        return CNS_ERR_NULL_PTR;
    const int64_t e = g->dtype == CNS_DT_F32 ? 4 : 2;
    if (off(g->rows_dev, e) || off(g->dy_dev, e) || off(g->drows_dev, e) || off(g->places_dev, 4) ||
        off(g->weights_dev, 4) || off(g->dweights_dev, 4) ||
        (g->drows_dev && (g->drows_dev == g->rows_dev || g->drows_dev == g->dy_dev)) ||
        (g->dweights_dev && g->dweights_dev == g->weights_dev))
        return CNS_ERR_INVALID_VALUE;
    p.rows = g->rows_dev;
    p.dy = g->dy_dev;
    p.places = g->places_dev;
    p.weights = g->weights_dev;
    p.drows = g->drows_dev;
    p.dweights = g->dweights_dev;
    p.tokens = g->tokens;
    p.limit = row_limit(g->rows);
    p.top_k = g->top_k;
    uint64_t bits = address(p.dy) | (g->width * e) | (p.dy_stride * e);
    if (p.dweights)
        bits |= address(p.rows) | (p.rows_stride * e);
    if (p.drows)
        bits |= address(p.drows) | (p.drows_stride * e);
    const int access = access_bytes(bits);
    p.units = static_cast<uint32_t>(g->width * e / access);
    DeviceInfo dev;
    if (int rc = current_device(&dev))
        return rc;
    if (p.tokens == 0)
        return CNS_SUCCESS;
    cudaStream_t s = to_stream(g->stream);
    CNS_CUDA(g->dtype == CNS_DT_F32    ? launch_combine_backward<CNS_DT_F32>(p, access, s)
             : g->dtype == CNS_DT_BF16 ? launch_combine_backward<CNS_DT_BF16>(p, access, s)
                                       : launch_combine_backward<CNS_DT_F16>(p, access, s));
    return CNS_SUCCESS;
}
