// route.cu -- routing tokens to experts (cns_route) and its gradient
// (cns_route_backward).
//
// One warp takes one token: lane l holds experts l * V .. l * V + V - 1 (V a
// power of two with 32 * V >= experts), so "lower index first" is "lower lane
// first, then lower element".
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "cns.h"
#include "cns_host.h"
#include "step_device.cuh"

namespace cns {
namespace {

constexpr int kWarps = 8;   // tokens of a CTA at a time

struct RouteParams {
    const void *logits;
    const float *bias;
    int32_t *ids;
    float *weights;
    float *scores;
    int32_t *offsets;
    int32_t *order;
    int32_t *places;
    int64_t tokens;
    int64_t stride;
    int32_t experts, top_k, score, groups, top_groups, group_top, renorm;
    float scale;
};

// Floats as integers in the same order: NaN above inf, -0 as 0, 0 for masked.
__device__ __forceinline__ uint32_t choice_key(float v)
{
    v += 0.f;   // -0 and 0 are equal
    const uint32_t u = __float_as_uint(v);
    if (v != v)
        return 0xffffffffu;
    if (u == 0xff800000u)
        return 0u;
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kFullWarp, v, d));
    return v;
}

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

template <int D, int V>
__global__ void __launch_bounds__(kWarps * 32) route_choose_kernel(const RouteParams p)
{
    using T = typename Elem<D>::type;
    extern __shared__ float s_value[];   // [kWarps][experts], with groups
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < p.tokens;
         t += static_cast<int64_t>(gridDim.x) * kWarps) {
        const T *row = static_cast<const T *>(p.logits) + t * p.stride;
        float x[V], s[V];
        uint32_t key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            x[i] = e < p.experts ? Elem<D>::get(row[e]) : -INFINITY;
        }
        row_scores<V>(x, s, p.score);
        if (p.scores) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane * V + i < p.experts)
                    p.scores[t * p.experts + lane * V + i] = s[i];
        }
        const bool by_logit = !p.bias && p.group_top == 1;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            float v = by_logit ? x[i] : s[i];
            if (p.bias && e < p.experts)
                v += p.bias[e];
            if (x[i] == -INFINITY)
                v = -INFINITY;
            key[i] = choice_key(v);
            if (p.groups > 1 && e < p.experts)
                s_value[warp * p.experts + e] = v;
        }
        if (p.groups > 1) {
            __syncwarp();
            // lane g: what group g is worth
            const int size = p.experts / p.groups;
            uint32_t worth = 0;
            if (lane < p.groups) {
                const float *v = s_value + warp * p.experts + lane * size;
                float a = -INFINITY, b = -INFINITY;   // the two best
                for (int i = 0; i < size; ++i) {
                    const float c = v[i];
                    if (choice_key(c) > choice_key(a)) {
                        b = a;
                        a = c;
                    } else if (choice_key(c) > choice_key(b)) {
                        b = c;
                    }
                }
                worth = choice_key(p.group_top == 2 && b != -INFINITY ? a + b : a);
            }
            int before = 0;   // groups that go before this one
            for (int g = 0; g < p.groups; ++g) {
                const uint32_t o = __shfl_sync(kFullWarp, worth, g);
                before += (o > worth || (o == worth && g < lane)) ? 1 : 0;
            }
            const uint32_t kept = __ballot_sync(kFullWarp, lane < p.groups && before < p.top_groups);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane * V + i;
                if (e < p.experts && !((kept >> (e / size)) & 1u))
                    key[i] = 0u;
            }
            __syncwarp();
        }
        // the top_k best; lane j keeps place j
        int my_id = -1;
        float my_x = -INFINITY, my_s = 0.f;
        for (int j = 0; j < p.top_k; ++j) {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                best = max(best, key[i]);
            const uint32_t top = __reduce_max_sync(kFullWarp, best);
            if (top == 0u)
                break;
            const int from = __ffs(__ballot_sync(kFullWarp, best == top)) - 1;
            int e = 0;
            float ex = 0.f, es = 0.f;
            if (lane == from) {
                bool found = false;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (!found && key[i] == top) {
                        found = true;
                        key[i] = 0u;
                        e = lane * V + i;
                        ex = x[i];
                        es = s[i];
                    }
                }
            }
            e = __shfl_sync(kFullWarp, e, from);
            ex = __shfl_sync(kFullWarp, ex, from);
            es = __shfl_sync(kFullWarp, es, from);
            if (lane == j) {
                my_id = e;
                my_x = ex;
                my_s = es;
            }
        }
        float w = my_s;
        if (p.renorm) {
            if (p.score == CNS_SCORE_SOFTMAX)
                row_scores<1>(&my_x, &w, CNS_SCORE_SOFTMAX);
            else
                w = my_s / (warp_sum(my_s) + 1e-20f);
        }
        if (lane < p.top_k) {
            p.ids[t * p.top_k + lane] = my_id;
            p.weights[t * p.top_k + lane] = my_id < 0 ? 0.f : w * p.scale;
        }
    }
}

// The plan, one CTA per expert: count the entries of lower experts (where
// this expert's list starts) and its own, then place its own in order.
__global__ void __launch_bounds__(256) route_place_kernel(const RouteParams p)
{
    __shared__ int s_count[8], s_lower[8];
    const int e = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n = p.tokens * p.top_k;
    int lower = 0, own = 0;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
        const int id = p.ids[i];
        lower += id >= 0 && id < e;
        own += id == e;
    }
    lower = __reduce_add_sync(kFullWarp, lower);
    own = __reduce_add_sync(kFullWarp, own);
    if (lane == 0) {
        s_lower[warp] = lower;
        s_count[warp] = own;
    }
    __syncthreads();
    lower = own = 0;
    for (int w = 0; w < 8; ++w) {
        lower += s_lower[w];
        own += s_count[w];
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        p.offsets[e] = lower;
        if (e == p.experts - 1)
            p.offsets[p.experts] = lower + own;
    }
    int at = lower;
    for (int64_t first = 0; first < n; first += blockDim.x) {
        const int64_t i = first + threadIdx.x;
        const bool mine = i < n && p.ids[i] == e;
        const uint32_t m = __ballot_sync(kFullWarp, mine);
        if (lane == 0)
            s_count[warp] = __popc(m);
        __syncthreads();
        int here = at, all = 0;
        for (int w = 0; w < 8; ++w) {
            if (w < warp)
                here += s_count[w];
            all += s_count[w];
        }
        if (mine) {
            const int place = here + __popc(m & ((1u << lane) - 1u));
            p.order[place] = static_cast<int32_t>(i);
            if (p.places)
                p.places[i] = place;
        }
        at += all;
        __syncthreads();
    }
    if (e == p.experts - 1) {
        // the rest of order, and the places without an expert
        for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
            if (i >= at)
                p.order[i] = -1;
            if (p.places && p.ids[i] < 0)
                p.places[i] = -1;
        }
    }
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

template <int D> struct LaunchChoose {
    const RouteParams &p;
    int grid;
    size_t smem;
    cudaStream_t s;
    template <int V> void operator()() { route_choose_kernel<D, V><<<grid, kWarps * 32, smem, s>>>(p); }
};

template <int D> struct LaunchBackward {
    const RouteGradParams &p;
    int grid;
    cudaStream_t s;
    template <int V> void operator()() { route_backward_kernel<D, V><<<grid, kWarps * 32, 0, s>>>(p); }
};

size_t workspace_bytes(int64_t, int32_t, int32_t) { return CNS_STEP_WORKSPACE_HEADER_BYTES; }

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
    p.score = r->score;
    p.groups = groups;
    p.top_groups = top_groups;
    p.group_top = r->group_top ? r->group_top : 1;
    p.renorm = r->renorm;
    p.scale = r->scale;
    const int grid = static_cast<int>(std::min<int64_t>((r->tokens + kWarps - 1) / kWarps, dev.sm_count * 8));
    const size_t smem = groups > 1 ? sizeof(float) * kWarps * r->experts : 0;
    if (grid > 0) {
        switch (r->dtype) {
        case CNS_DT_F32: by_width(r->experts, LaunchChoose<CNS_DT_F32>{p, grid, smem, s}); break;
        case CNS_DT_BF16: by_width(r->experts, LaunchChoose<CNS_DT_BF16>{p, grid, smem, s}); break;
        default: by_width(r->experts, LaunchChoose<CNS_DT_F16>{p, grid, smem, s}); break;
        }
    }
    if (plan)
        route_place_kernel<<<r->experts, 256, 0, s>>>(p);
    CNS_CUDA(cudaGetLastError());
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
