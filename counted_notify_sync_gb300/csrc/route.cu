// route.cu -- routing tokens to experts (cns_route) and its gradient
// (cns_route_backward).
//
// The entry points, the kernels of the plan and of the gradient.  The routing
// kernel is in route_kernels.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "cns.h"
#include "cns_host.h"
#include "route_kernels.cuh"

namespace cns {
namespace {

constexpr int kPlanHeld = 4;   // batches of a warp's tokens whose ids stay in registers

// The plan of a routing by several CTAs: a grid of its own, as large as the one that chose.  Its CTAs set up while
// that one's last are still choosing.
__global__ void __launch_bounds__(kRouteWarps * 32, 1) route_plan_kernel(const __grid_constant__ RouteParams p)
{
    extern __shared__ uint32_t smem[];
    __shared__ int s_stop;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int E = p.experts, e = threadIdx.x;
    const uint32_t cta = blockIdx.x, ctas = gridDim.x;
    const Stretch mine(p.tokens, warp, warps);
    const int seg = place_lanes(p), per = 32 / seg, place = lane & (seg - 1);
    uint32_t *s_count = smem;
    for (int i = threadIdx.x; i < warps * E; i += blockDim.x)
        s_count[i] = 0u;
    __syncthreads();
    grid_dependency_wait();   // all choices, and all CTAs' counts
    // all loads before the first use of any: the workspace's status, the ids of the warp's first batches of tokens,
    // the sums of the blocks and the counts of the CTA's block for expert e
    const bool stop = threadIdx.x == 0 && ld_relaxed_gpu(p.header + kStepStatusWord + 1) != 0u;   // an earlier call failed
    auto id_of = [&](int64_t t) { return t < mine.last && place < p.top_k ? p.ids[t * p.top_k + place] : -1; };
    int held[kPlanHeld];
    int64_t t = mine.first + lane / seg;
#pragma unroll
    for (int i = 0; i < kPlanHeld; ++i, t += per)
        held[i] = id_of(t);
    uint32_t before = 0, total = 0;
    if (e < E) {
        constexpr uint32_t kBlocks = kStepMaxCtas / kStepBlockCtas;
        const uint32_t block = cta / kStepBlockCtas, *counts = p.counts + e;
        uint32_t c[kBlocks], r[kStepBlockCtas];
#pragma unroll
        for (uint32_t i = 0; i < kBlocks; ++i)
            c[i] = i * kStepBlockCtas < ctas ? __ldcg(block_sums(p, i) + e) : 0u;
#pragma unroll
        for (uint32_t i = 0; i < kStepBlockCtas; ++i)
            r[i] = block * kStepBlockCtas + i < cta ? __ldcg(counts + (block * kStepBlockCtas + i) * E) : 0u;
#pragma unroll
        for (uint32_t i = 0; i < kBlocks; ++i) {
            total += c[i];
            before += i < block ? c[i] : 0u;
        }
#pragma unroll
        for (uint32_t i = 0; i < kStepBlockCtas; ++i)
            before += r[i];
    }
#pragma unroll
    for (int i = 0; i < kPlanHeld; ++i)
        if (held[i] >= 0)
            atomicAdd(&s_count[warp * E + held[i]], 1u);
    for (; t - lane / seg < mine.last; t += per) {
        const int id = id_of(t);
        if (id >= 0)
            atomicAdd(&s_count[warp * E + id], 1u);
    }
    if (threadIdx.x == 0)
        s_stop = stop;
    __syncthreads();
    if (s_stop)
        return;
    // every CTA has the sums when the last one says so; it clears them (and the count of those that said so)
    uint32_t earlier = 0;
    if (threadIdx.x == 0) {
        fence_release_gpu();
        earlier = atom_add_relaxed_gpu(p.header + kStepPlanWord, 1u);
    }
    place_entries(p, mine, held, before, total, s_count, s_count + warps * E, s_count + (warps + 1) * E);
    if (warp == 0 && __shfl_sync(kFullWarp, earlier, 0) == ctas - 1u) {
        fence_acquire_gpu();
        for (uint32_t i = lane; i < kStepSumWords / 4; i += 32)
            reinterpret_cast<uint4 *>(block_sums(p, 0u))[i] = make_uint4(0u, 0u, 0u, 0u);
        if (lane == 0)
            st_relaxed_gpu(p.header + kStepPlanWord, 0u);
    }
}

cudaError_t launch_plan(const RouteParams &p, int ctas, int warps, cudaStream_t s)
{
    const size_t smem = plan_smem(p.experts, warps);
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(route_plan_kernel), smem,
                                     plan_smem(CNS_ROUTE_MAX_EXPERTS, kRouteWarps));
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = early_launch(&attr);
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, route_plan_kernel, p);
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

// What of a row has a gradient: the chosen experts alone; every expert through
// the softmax (weights that are not renormalised); every expert through dscores.
enum : int { kGradSparse = 0, kGradSoftmax = 1, kGradScores = 2 };

constexpr int kGradWarps = 8;
constexpr int kHeld = 32;   // elements of a row that a lane keeps in registers

template <int SEG>
__device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int d = SEG / 2; d > 0; d >>= 1)
        v += __shfl_xor_sync(kFullWarp, v, d);
    return v;
}

template <int SEG>
__device__ __forceinline__ float lanes_max(float v)
{
#pragma unroll
    for (int d = SEG / 2; d > 0; d >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kFullWarp, v, d));
    return v;
}

// W elements in a row; 16 bytes of them or more at once, or one.
template <int D, int W>
__device__ __forceinline__ void load_elems(const typename Elem<D>::type *a, float *v)
{
    using T = typename Elem<D>::type;
    if constexpr (W == 1) {
        v[0] = Elem<D>::get(*a);
    } else {
        constexpr int N = 16 / static_cast<int>(sizeof(T));   // of a vector
#pragma unroll
        for (int j = 0; j < W; j += N) {
            const uint4 u = *reinterpret_cast<const uint4 *>(a + j);
            const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[j + i] = Elem<D>::get(e[i]);
        }
    }
}

template <int D, int W>
__device__ __forceinline__ void store_elems(typename Elem<D>::type *a, const float *v)
{
    using T = typename Elem<D>::type;
    if constexpr (W == 1) {
        *a = Elem<D>::put(v[0]);
    } else {
        static_assert(W * sizeof(T) == 16, "one vector");
        uint4 u;
        T *e = reinterpret_cast<T *>(&u);
#pragma unroll
        for (int i = 0; i < W; ++i)
            e[i] = Elem<D>::put(v[i]);
        *reinterpret_cast<uint4 *>(a) = u;
    }
}

// dL/dlogits.  With g_j = scale * dL/dw_j at the chosen experts, h = dL/ds, s
// the scores and S their sum over the chosen:
//   softmax             p_e (h_e + g_e - sum_i p_i (h_i + g_i))
//   softmax, renorm     p_e (h_e - sum_i p_i h_i), and q_j (g_j - sum_i q_i g_i)
//                       at the chosen, q the softmax over the chosen
//   sigmoid             s (1 - s) (h + g)
//   sigmoid, renorm     the same with g_j replaced by (g_j - sum_i g_i s_i / S) / S
// So a row is what holds for experts that were not chosen (without h, and unless
// the gradient goes through the whole softmax, 0), with the chosen ones'
// written over it.
//
// Bound by the bytes of dlogits, and of logits where the whole softmax takes
// part.  SEG lanes take a token (8 for up to 8 places, so a warp has four
// tokens and its reductions serve them together), W elements of 16 bytes a
// lane; each lane also has one place.  For the softmax a row of up to HOLD
// vectors a lane stays in registers, longer ones (and rows at odd addresses) are
// read from L1 a second and a third time, and their exponentials taken twice:
// 50021 x 160 f32 13.8 us (4.8 TB/s) held, 18.1 us read again.  The sparse forms
// write zeros and the chosen ones: 16384 x 256 f32 4.5 us of the GPU (4.1 TB/s).
// Exponentials are expf: by ex2.approx of a rounded product the first took 13.4
// us, and gradients far below the row's largest were off by up to 4e-6 of
// themselves; now they are within 1.9e-6.
template <int D, int W, int SEG, int HOLD, int MODE>
__global__ void __launch_bounds__(kGradWarps * 32, MODE == kGradSparse ? 8 : 4) route_backward_kernel(const RouteGradParams p)
{
    using T = typename Elem<D>::type;
    const int lane = threadIdx.x & 31, place = lane & (SEG - 1);
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kGradWarps * 32 / SEG);
    const int64_t begin = (static_cast<int64_t>(blockIdx.x) * kGradWarps + (threadIdx.x >> 5)) * (32 / SEG);
    const bool softmax = MODE == kGradSoftmax || p.score == CNS_SCORE_SOFTMAX;
    const bool renorm = MODE != kGradSoftmax && p.renorm;
    constexpr bool whole = MODE != kGradSparse;
    static_assert(HOLD == 0 || MODE == kGradSoftmax, "only a row that is read again is held");
    grid_dependency_wait();   // launched early: nothing of the tensors before this
    for (int64_t t0 = begin; t0 < p.tokens; t0 += step) {
        const int64_t t = t0 + lane / SEG;
        const bool token = t < p.tokens;
        const T *row = static_cast<const T *>(p.logits) + t * p.stride;
        const float *ds = MODE == kGradScores ? p.dscores + t * p.experts : nullptr;
        T *out = static_cast<T *>(p.dlogits) + t * p.dstride;
        float held[HOLD ? HOLD : 1][W];   // the lane's logits, then e^(x - top)
        if (HOLD) {
#pragma unroll
            for (int j = 0; j < HOLD; ++j) {
                const int e = (j * SEG + place) * W;
#pragma unroll
                for (int i = 0; i < W; ++i)
                    held[j][i] = -INFINITY;
                if (token && e < p.experts)
                    load_elems<D, W>(row + e, held[j]);
            }
        }
        // the lane's place
        int id = token && place < p.top_k ? p.ids[t * p.top_k + place] : -1;
        if (id >= p.experts)
            id = -1;
        const bool there = id >= 0;
        float g = there ? p.dweights[t * p.top_k + place] * p.scale : 0.f;
        const float x = there ? Elem<D>::get(row[id]) : -INFINITY;
        const float h = MODE == kGradScores && there ? ds[id] : 0.f;

        // the row's softmax: top and the sum under it, and sum_i e^(x_i - top) h_i
        float top = 0.f, sum = 1.f, mean = 0.f;
        if (whole && softmax) {
            top = -INFINITY;
            if constexpr (HOLD > 0) {
#pragma unroll
                for (int j = 0; j < HOLD; ++j)
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        top = fmaxf(top, held[j][i]);
            } else if (token) {
#pragma unroll 4
                for (int e = place * W; e < p.experts; e += SEG * W) {
                    float v[W];
                    load_elems<D, W>(row + e, v);
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        top = fmaxf(top, v[i]);
                }
            }
            top = lanes_max<SEG>(top);
            if (top == -INFINITY)
                top = 0.f;   // every expert masked
            sum = 0.f;
            if constexpr (HOLD > 0) {
#pragma unroll
                for (int j = 0; j < HOLD; ++j) {
                    if (j * SEG * W >= p.experts)
                        break;   // no lane has any (an expf takes 8 instructions)
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        held[j][i] = expf(held[j][i] - top);
                        sum += held[j][i];
                    }
                }
            } else if (token) {
#pragma unroll 4
                for (int e = place * W; e < p.experts; e += SEG * W) {
                    float v[W], w[W];
                    load_elems<D, W>(row + e, v);
                    if (MODE == kGradScores)
                        load_elems<CNS_DT_F32, W>(ds + e, w);
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const float ex = expf(v[i] - top);
                        sum += ex;
                        if (MODE == kGradScores)
                            mean = fmaf(ex, w[i], mean);
                    }
                }
            }
            sum = lanes_sum<SEG>(sum);
            if (sum == 0.f)
                sum = 1.f;
            mean = lanes_sum<SEG>(mean) / sum;
        }

        // the chosen ones' values
        float d;
        if (softmax) {
            const float pj = whole && there ? expf(x - top) / sum : 0.f;
            if (renorm) {
                const float best = lanes_max<SEG>(x);
                float q = there ? expf(x - best) : 0.f;
                q = q / lanes_sum<SEG>(q);
                const float inner = lanes_sum<SEG>(there ? q * g : 0.f);
                d = q * (g - inner) + pj * (h - mean);
            } else {
                mean += lanes_sum<SEG>(pj * g);
                d = pj * (h + g - mean);
            }
        } else {
            const float ex = expf(-fabsf(x)), r = 1.f / (1.f + ex);   // s and 1 - s without cancellation
            const float s = there ? (x >= 0.f ? r : ex * r) : 0.f, rest = x >= 0.f ? ex * r : r;
            if (renorm) {
                const float total = lanes_sum<SEG>(s) + 1e-20f;
                g = (g - lanes_sum<SEG>(g * s) / total) / total;
            }
            d = s * rest * (h + g);
        }

        // the row, then the chosen ones over it
        if (token) {
            const float scale = 1.f / sum;
            // one vector: its logits, or e^(x - top) of them, become its gradient
            auto finish = [&](int e, float *v, bool exps) {
                float w[W];
                if (MODE == kGradScores)
                    load_elems<CNS_DT_F32, W>(ds + e, w);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    if (!whole) {
                        v[i] = 0.f;
                    } else if (softmax) {
                        v[i] = (exps ? v[i] : expf(v[i] - top)) * scale * ((MODE == kGradScores ? w[i] : 0.f) - mean);
                    } else {
                        const float ex = expf(-fabsf(v[i])), r = 1.f / (1.f + ex);
                        v[i] = r * (ex * r) * w[i];
                    }
                }
                store_elems<D, W>(out + e, v);
            };
            if constexpr (HOLD > 0) {
#pragma unroll
                for (int j = 0; j < HOLD; ++j) {
                    const int e = (j * SEG + place) * W;
                    if (e < p.experts)
                        finish(e, held[j], true);
                }
            } else {
#pragma unroll 4
                for (int e = place * W; e < p.experts; e += SEG * W) {
                    float v[W];
                    if (whole)
                        load_elems<D, W>(row + e, v);
                    finish(e, v, false);
                }
            }
        }
        __syncwarp();   // orders the lanes' stores to one place
        if (there)
            out[id] = Elem<D>::put(d);
    }
}

template <int D>
cudaError_t launch_backward(const RouteGradParams &p, int sms, cudaStream_t s)
{
    using T = typename Elem<D>::type;
    constexpr int W = 16 / static_cast<int>(sizeof(T));
    const auto whole16 = [](const void *a) { return reinterpret_cast<uintptr_t>(a) % 16 == 0; };
    // whole vectors in every row
    const bool wide = p.experts % W == 0 && whole16(p.logits) && whole16(p.dlogits) && whole16(p.dscores) &&
                      p.stride % W == 0 && p.dstride % W == 0;
    const auto launch = [&](auto kernel, int seg) {
        const int64_t per = kGradWarps * (32 / seg), ctas = (p.tokens + per - 1) / per;
        cudaLaunchAttribute early;
        cudaLaunchConfig_t cfg = early_launch(&early);
        cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(ctas, static_cast<int64_t>(sms) * 128)));
        cfg.blockDim = dim3(kGradWarps * 32);
        cfg.stream = s;
        RouteGradParams arg = p;
        void *args[] = {&arg};
        return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(kernel), args);
    };
    const bool eight = p.top_k <= 8;
    if (p.dscores)
        return wide && eight ? launch(route_backward_kernel<D, W, 8, 0, kGradScores>, 8)
               : wide        ? launch(route_backward_kernel<D, W, 32, 0, kGradScores>, 32)
                             : launch(route_backward_kernel<D, 1, 32, 0, kGradScores>, 32);
    if (p.score == CNS_SCORE_SOFTMAX && !p.renorm)
        return wide && eight && p.experts <= kHeld * 8 ? launch(route_backward_kernel<D, W, 8, kHeld / W, kGradSoftmax>, 8)
               : wide && eight                         ? launch(route_backward_kernel<D, W, 8, 0, kGradSoftmax>, 8)
               : wide ? launch(route_backward_kernel<D, W, 32, 16 / W, kGradSoftmax>, 32)
                      : launch(route_backward_kernel<D, 1, 32, 0, kGradSoftmax>, 32);
    return wide && eight ? launch(route_backward_kernel<D, W, 8, 0, kGradSparse>, 8)
           : wide        ? launch(route_backward_kernel<D, W, 32, 0, kGradSparse>, 32)
           : eight       ? launch(route_backward_kernel<D, 1, 8, 0, kGradSparse>, 8)
                         : launch(route_backward_kernel<D, 1, 32, 0, kGradSparse>, 32);
}

size_t workspace_bytes(int64_t, int32_t experts, int32_t)
{
    return CNS_STEP_WORKSPACE_HEADER_BYTES + sizeof(uint32_t) * kStepMaxCtas * static_cast<size_t>(experts);
}

// Up to kOneCtaTokens one CTA routes them all, in one launch (32 x 64 5.4 us against 6.9 us by eight CTAs; 32 x 256
// 10.2 against 9.8, 64 x 256 15.9 against 10.1).  More tokens go to as many CTAs as there are SMs, if each has
// kLeastTokens: a warp alone is latency, and more warps to an SM slow one another (512 x 256 10.6 us, with eight
// tokens a CTA 12.0, with 32 13.0; 3001 x 160 11.3 us on 152 CTAs, 11.5 on 94).
constexpr int64_t kOneCtaTokens = 32, kLeastTokens = 4;

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
    p.key_step = 512u;
    p.header = static_cast<uint32_t *>(r->workspace_dev);
    p.counts = p.header + CNS_STEP_WORKSPACE_HEADER_BYTES / 4;
    if (r->tokens > 0 || plan) {
        int ctas, warps;
        if (r->tokens <= kOneCtaTokens) {
            ctas = 1;
            warps = static_cast<int>(std::min<int64_t>(kRouteWarps, std::max<int64_t>(r->tokens, 4)));
        } else {
            ctas = static_cast<int>(std::min<int64_t>((r->tokens + kLeastTokens - 1) / kLeastTokens,
                                                      std::min<int>(dev.sm_count, kStepMaxCtas)));
            warps = kRouteWarps;
        }
        const bool by_score = p.bias || p.group_top == 2;
        const auto launch = r->dtype == CNS_DT_F32    ? (by_score ? launch_route_f32_score : launch_route_f32_logit)
                            : r->dtype == CNS_DT_BF16 ? (by_score ? launch_route_bf16_score : launch_route_bf16_logit)
                                                      : (by_score ? launch_route_f16_score : launch_route_f16_logit);
        CNS_CUDA(launch(p, ctas, warps, s));
        if (plan && ctas > 1) {
            const cudaError_t e = launch_plan(p, ctas, warps, s);
            if (e != cudaSuccess) {
                // nobody will take up what the first grid adds to the blocks' sums: later plans must not
                (void)cudaGetLastError();
                (void)cudaMemsetAsync(p.header + kStepSumWord, 0, kStepSumWords * sizeof(uint32_t), s);
                return cuda_fail(e, "routing plan launch");
            }
        }
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
    CNS_CUDA(g->dtype == CNS_DT_F32    ? launch_backward<CNS_DT_F32>(p, dev.sm_count, s)
             : g->dtype == CNS_DT_BF16 ? launch_backward<CNS_DT_BF16>(p, dev.sm_count, s)
                                       : launch_backward<CNS_DT_F16>(p, dev.sm_count, s));
    return CNS_SUCCESS;
}
