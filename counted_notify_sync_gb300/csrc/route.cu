// route.cu -- routing tokens to experts (cns_route) and its gradient
// (cns_route_backward).
//
// The entry points, and the gradient's kernel: one warp takes one token, lane l
// holds experts l * V .. l * V + V - 1.  The routing kernel is in
// route_kernels.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "cns.h"
#include "cns_host.h"
#include "route_kernels.cuh"

namespace cns {
namespace {

constexpr int kWarps = 8;   // tokens of a CTA at a time

// Scores of the warp's row: sigmoid, or softmax over the row.  A row without
// an unmasked logit scores 0.
template <int V>
__device__ __forceinline__ void row_scores(const float *x, float *s, int score)
{
    if (score == CNS_SCORE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            s[i] = 1.f / (1.f + expf(-x[i]));
        return;
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i)
        top = fmaxf(top, x[i]);
    top = warp_max(top);
    if (top == -INFINITY)
        top = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s[i] = expf(x[i] - top);
        sum += s[i];
    }
    sum = warp_sum(sum);
    if (sum == 0.f)
        sum = 1.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        s[i] = s[i] / sum;
}

struct RouteGradParams {
    const void *logits;
    const int32_t *ids;
    const float *dweights;
    const float *dscores;
    void *dlogits;
    int64_t tokens, stride, dstride;
    int32_t experts, top_k, score, renorm;
    float scale;
};

// dL/dlogits of one token per warp.  With g_j = scale * dL/dw_j at the chosen
// experts, s the scores and S their sum over the chosen:
//   softmax             p_e (h_e - sum_i p_i h_i), h = g at the chosen + dL/ds
//   softmax, renorm     q_j (g_j - sum_i q_i g_i) at the chosen, q the softmax
//                       over the chosen; and the line above for dL/ds alone
//   sigmoid             s (1 - s) h
//   sigmoid, renorm     the same with g_j replaced by (g_j - sum_i g_i s_i / S) / S
template <int D, int V>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(const RouteGradParams p)
{
    using T = typename Elem<D>::type;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < p.tokens;
         t += static_cast<int64_t>(gridDim.x) * kWarps) {
        const T *row = static_cast<const T *>(p.logits) + t * p.stride;
        T *out = static_cast<T *>(p.dlogits) + t * p.dstride;
        int id = -1;
        float g = 0.f, gx = -INFINITY;
        if (lane < p.top_k) {
            id = p.ids[t * p.top_k + lane];
            if (id >= p.experts)
                id = -1;
            if (id >= 0) {
                g = p.dweights[t * p.top_k + lane] * p.scale;
                gx = Elem<D>::get(row[id]);
            }
        }
        float x[V], s[V], h[V];
        const bool whole = p.dscores || (p.score == CNS_SCORE_SOFTMAX && !p.renorm);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            x[i] = whole && e < p.experts ? Elem<D>::get(row[e]) : -INFINITY;
            h[i] = p.dscores && e < p.experts ? p.dscores[t * p.experts + e] : 0.f;
        }
        float d = 0.f;   // the chosen expert's own part
        bool spread = false;   // g joins h before the product with the score
        if (p.score == CNS_SCORE_SOFTMAX) {
            if (p.renorm) {
                float q;
                row_scores<1>(&gx, &q, CNS_SCORE_SOFTMAX);
                d = q * (g - warp_sum(g * q));
            } else {
                spread = true;
            }
        } else {
            const float e = expf(-fabsf(gx)), r = 1.f / (1.f + e);   // s and 1 - s without cancellation
            const float sc = gx >= 0.f ? r : e * r, co = gx >= 0.f ? e * r : r;
            const float sg = id >= 0 ? sc : 0.f;
            if (p.renorm) {
                const float sum = warp_sum(sg) + 1e-20f;
                g = (g - warp_sum(g * sg) / sum) / sum;
            }
            d = id >= 0 ? g * sg * co : 0.f;
        }
        if (whole) {
            if (spread) {
                for (int j = 0; j < p.top_k; ++j) {
                    const int e = __shfl_sync(kFullWarp, id, j);
                    const float v = __shfl_sync(kFullWarp, g, j);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        h[i] += lane * V + i == e ? v : 0.f;
                }
            }
            if (p.score == CNS_SCORE_SOFTMAX) {
                row_scores<V>(x, s, CNS_SCORE_SOFTMAX);
                float mean = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    mean += s[i] != 0.f ? s[i] * h[i] : 0.f;
                mean = warp_sum(mean);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    h[i] = s[i] != 0.f ? s[i] * (h[i] - mean) : 0.f;
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float e = expf(-fabsf(x[i])), r = 1.f / (1.f + e);
                    h[i] = h[i] * r * (e * r);
                }
            }
        }
        if (!spread) {
            for (int j = 0; j < p.top_k; ++j) {
                const int e = __shfl_sync(kFullWarp, id, j);
                const float v = __shfl_sync(kFullWarp, d, j);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    h[i] += lane * V + i == e ? v : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane * V + i < p.experts)
                out[lane * V + i] = Elem<D>::put(h[i]);
    }
}

// Calls f.template operator()<V>() for the smallest V with 32 * V >= experts.
template <class F>
void by_width(int experts, F f)
{
    if (experts <= 32)
        f.template operator()<1>();
    else if (experts <= 64)
        f.template operator()<2>();
    else if (experts <= 128)
        f.template operator()<4>();
    else if (experts <= 256)
        f.template operator()<8>();
    else
        f.template operator()<16>();
}

template <int D> struct LaunchBackward {
    const RouteGradParams &p;
    int grid;
    cudaStream_t s;
    template <int V> void operator()() { route_backward_kernel<D, V><<<grid, kWarps * 32, 0, s>>>(p); }
};

size_t workspace_bytes(int64_t, int32_t experts, int32_t)
{
    return CNS_STEP_WORKSPACE_HEADER_BYTES + sizeof(uint32_t) * kStepMaxCtas * static_cast<size_t>(experts);
}

// Up to this many tokens one CTA routes them all and needs no exchange.
constexpr int64_t kOneCtaTokens = 64;

bool sizes_ok(int64_t tokens, int32_t experts, int32_t top_k)
{
    return tokens >= 0 && experts >= 1 && experts <= CNS_ROUTE_MAX_EXPERTS && top_k >= 1 &&
           top_k <= CNS_ROUTE_MAX_TOP_K && top_k <= experts && tokens <= 0x7fffffff / top_k;
}

bool off_element(const void *p, int32_t dtype)
{
    return reinterpret_cast<uintptr_t>(p) % (dtype == CNS_DT_F32 ? 4 : 2) != 0;
}

bool off_word(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 != 0; }

}  // namespace
}  // namespace cns

using namespace cns;

extern "C" int cns_route_workspace_bytes(int64_t tokens, int32_t experts, int32_t top_k, size_t *bytes)
{
    if (!bytes)
        return CNS_ERR_NULL_PTR;
    if (!sizes_ok(tokens, experts, top_k))
        return CNS_ERR_INVALID_VALUE;
    *bytes = workspace_bytes(tokens, experts, top_k);
    return CNS_SUCCESS;
}

extern "C" int cns_route(cns_route_t *r)
{
    TraceRange tr("cns_route", r ? static_cast<uint64_t>(r->tokens) : 0);
    if (!r)
        return CNS_ERR_NULL_PTR;
    if (!sizes_ok(r->tokens, r->experts, r->top_k) || r->dtype < CNS_DT_F32 || r->dtype > CNS_DT_F16 ||
        (r->score != CNS_SCORE_SIGMOID && r->score != CNS_SCORE_SOFTMAX) || !std::isfinite(r->scale) ||
        r->renorm < 0 || r->renorm > 1 || r->group_top < 0 || r->group_top > 2)
        return CNS_ERR_INVALID_VALUE;
    const int groups = r->groups ? r->groups : 1, top_groups = r->top_groups ? r->top_groups : groups;
    if (groups < 1 || groups > CNS_ROUTE_MAX_GROUPS || r->experts % groups || top_groups < 1 || top_groups > groups ||
        r->top_k > r->experts / groups * top_groups)
        return CNS_ERR_INVALID_VALUE;
    const int64_t stride = r->logits_stride ? r->logits_stride : r->experts;
    if (stride < r->experts)
        return CNS_ERR_INVALID_VALUE;
    const bool plan = r->offsets_dev != nullptr;
    if (!plan && (r->order_dev || r->places_dev))
        return CNS_ERR_INVALID_VALUE;
    if (plan && (!r->workspace_dev || (r->tokens > 0 && !r->order_dev)))
        return CNS_ERR_NULL_PTR;
    if (r->tokens > 0 && (!r->logits_dev || !r->ids_dev || !r->weights_dev))
        return CNS_ERR_NULL_PTR;
    if (off_element(r->logits_dev, r->dtype) || off_word(r->bias_dev) || off_word(r->ids_dev) ||
        off_word(r->weights_dev) || off_word(r->scores_dev) || off_word(r->offsets_dev) || off_word(r->order_dev) ||
        off_word(r->places_dev))
        return CNS_ERR_INVALID_VALUE;
    if (plan && (reinterpret_cast<uintptr_t>(r->workspace_dev) % CNS_STEP_WORKSPACE_ALIGN ||
                 r->workspace_bytes < workspace_bytes(r->tokens, r->experts, r->top_k)))
        return CNS_ERR_INVALID_VALUE;
    DeviceInfo dev;
    if (int rc = current_device(&dev))
        return rc;
    cudaStream_t s = to_stream(r->stream);
    RouteParams p = {};
    p.logits = r->logits_dev;
    p.bias = r->bias_dev;
    p.ids = r->ids_dev;
    p.weights = r->weights_dev;
    p.scores = r->scores_dev;
    p.offsets = r->offsets_dev;
    p.order = r->order_dev;
    p.places = r->places_dev;
    p.tokens = r->tokens;
    p.stride = stride;
    p.experts = r->experts;
    p.top_k = r->top_k;
    p.softmax = r->score == CNS_SCORE_SOFTMAX;
    p.plan = plan;
    p.groups = groups;
    p.top_groups = top_groups;
    p.group_top = r->group_top ? r->group_top : 1;
    p.renorm = r->renorm;
    p.scale = r->scale;
    p.timeout_ns = barrier_timeout_ns(r->timeout_ms);
    p.header = static_cast<uint32_t *>(r->workspace_dev);
    p.counts = p.header + CNS_STEP_WORKSPACE_HEADER_BYTES / 4;
    if (r->tokens > 0 || plan) {
        int ctas, warps;
        if (r->tokens <= kOneCtaTokens) {
            ctas = 1;
            warps = static_cast<int>(std::min<int64_t>(kRouteWarps, std::max<int64_t>(r->tokens, 4)));
        } else {
            ctas = static_cast<int>(std::min<int64_t>((r->tokens + kRouteWarps - 1) / kRouteWarps,
                                                      std::min<int>(dev.sm_count, kStepMaxCtas)));
            warps = kRouteWarps;
        }
        const cudaError_t e = r->dtype == CNS_DT_F32    ? launch_route_f32(p, ctas, warps, s)
                              : r->dtype == CNS_DT_BF16 ? launch_route_bf16(p, ctas, warps, s)
                                                        : launch_route_f16(p, ctas, warps, s);
        if (e == cudaErrorCooperativeLaunchTooLarge) {
            (void)cudaGetLastError();
            return CNS_ERR_NOT_RESIDENT;
        }
        if (e != cudaSuccess)
            return cuda_fail(e, "route launch");
    }
    if (!r->sync)
        return CNS_SUCCESS;
    r->device_status = 0;
    if (!plan) {
        CNS_CUDA(cudaStreamSynchronize(s));
        return CNS_SUCCESS;
    }
    if (int rc = syncall_read_workspace(r->workspace_dev, r->stream, nullptr, nullptr, &r->device_status))
        return rc;
    return r->device_status;
}

extern "C" int cns_route_backward(const cns_route_grad_t *g)
{
    TraceRange tr("cns_route_backward", g ? static_cast<uint64_t>(g->tokens) : 0);
    if (!g)
        return CNS_ERR_NULL_PTR;
    if (!sizes_ok(g->tokens, g->experts, g->top_k) || g->dtype < CNS_DT_F32 || g->dtype > CNS_DT_F16 ||
        (g->score != CNS_SCORE_SIGMOID && g->score != CNS_SCORE_SOFTMAX) || !std::isfinite(g->scale) ||
        g->renorm < 0 || g->renorm > 1)
        return CNS_ERR_INVALID_VALUE;
    const int64_t stride = g->logits_stride ? g->logits_stride : g->experts;
    const int64_t dstride = g->dlogits_stride ? g->dlogits_stride : g->experts;
    if (stride < g->experts || dstride < g->experts)
        return CNS_ERR_INVALID_VALUE;
    if (g->tokens > 0 && (!g->logits_dev || !g->ids_dev || !g->dweights_dev || !g->dlogits_dev))
        return CNS_ERR_NULL_PTR;
    if (off_element(g->logits_dev, g->dtype) || off_element(g->dlogits_dev, g->dtype) || off_word(g->ids_dev) ||
        off_word(g->dweights_dev) || off_word(g->dscores_dev) ||
        (g->tokens > 0 && g->dlogits_dev == g->logits_dev))
        return CNS_ERR_INVALID_VALUE;
    DeviceInfo dev;
    if (int rc = current_device(&dev))
        return rc;
    if (g->tokens == 0)
        return CNS_SUCCESS;
    RouteGradParams p = {};
    p.logits = g->logits_dev;
    p.ids = g->ids_dev;
    p.dweights = g->dweights_dev;
    p.dscores = g->dscores_dev;
    p.dlogits = g->dlogits_dev;
    p.tokens = g->tokens;
    p.stride = stride;
    p.dstride = dstride;
    p.experts = g->experts;
    p.top_k = g->top_k;
    p.score = g->score;
    p.renorm = g->renorm;
    p.scale = g->scale;
    cudaStream_t s = to_stream(g->stream);
    const int grid = static_cast<int>(std::min<int64_t>((g->tokens + kWarps - 1) / kWarps, dev.sm_count * 8));
    switch (g->dtype) {
    case CNS_DT_F32: by_width(g->experts, LaunchBackward<CNS_DT_F32>{p, grid, s}); break;
    case CNS_DT_BF16: by_width(g->experts, LaunchBackward<CNS_DT_BF16>{p, grid, s}); break;
    default: by_width(g->experts, LaunchBackward<CNS_DT_F16>{p, grid, s}); break;
    }
    CNS_CUDA(cudaGetLastError());
    return CNS_SUCCESS;
}
