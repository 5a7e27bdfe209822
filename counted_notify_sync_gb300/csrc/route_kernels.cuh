// route_kernels.cuh -- the routing kernel: choose each token's experts, weigh
// them, and place the entries by expert.  One translation unit per element
// type of the logits (route_f32.cu, route_bf16.cu, route_f16.cu).
//
// One warp takes one token: element i of lane l is expert 32 i + l, so every
// load of a row is coalesced whatever its alignment, and among equal choice
// values the lower expert is the lower element, then the lower lane.
//
// Choice.  Each lane keeps the two best of its elements; a round takes the best
// of the lanes' heads with one redux, and the lane that had it moves its
// second one up.  A lane that gives a third one rescans its elements (a rare,
// warp-uniform branch), so a round costs a dozen instructions whatever the
// number of experts.
//
// Plan.  CTA b has a stretch of tokens and each of its warps a stretch of
// those, so that entries in order are warps in order.  Phase 1 chooses and
// counts per warp; the CTAs publish their counts per expert and meet
// (step_device.cuh's exchange as a barrier); every CTA sums the rows before
// its own, and phase 2 walks the tokens again in order, each entry's place
// being its expert's running count.  Only integer sums: the plan does not
// depend on timing.
#pragma once

#include "cns_host.h"
#include "step_device.cuh"

namespace cns {

constexpr int kRouteWarps = 32;   // of the largest CTA

struct RouteParams {
    const void *logits;
    const float *bias;
    int32_t *ids;
    float *weights;
    float *scores;
    int32_t *offsets;
    int32_t *order;
    int32_t *places;
    uint32_t *header;    // of the workspace
    uint32_t *counts;    // [CTAs][experts], in the workspace
    uint64_t timeout_ns;
    int64_t tokens;
    int64_t stride;
    int32_t experts, top_k, groups, top_groups, group_top;
    int32_t softmax, renorm, plan;
    float scale;
};

// Defined in the translation unit of each element type.
cudaError_t launch_route_f32(const RouteParams &p, int ctas, int warps, cudaStream_t s);
cudaError_t launch_route_bf16(const RouteParams &p, int ctas, int warps, cudaStream_t s);
cudaError_t launch_route_f16(const RouteParams &p, int ctas, int warps, cudaStream_t s);

#ifdef CNS_ROUTE_KERNELS

// Floats as integers in the same order.  The addition makes -0 a 0 and every
// NaN the positive one, which ends up above inf.
__device__ __forceinline__ uint32_t choice_key(float v)
{
    const uint32_t u = __float_as_uint(v + 0.f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
constexpr uint32_t kMaskedKey = 0x007fffffu;   // of -inf; what was taken has key 0

__device__ __forceinline__ float sigmoid_of(float x) { return 1.f / (1.f + expf(-x)); }

// The two best of a lane's elements that are not in `taken`, the lower
// element first among equals; key 0 where there is none.
struct Heads {
    uint32_t key1, key2;
    int i1, i2;
};

template <int V>
__device__ __forceinline__ Heads heads_of(const uint32_t *key, uint32_t taken)
{
    Heads h{0u, 0u, 0, 0};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t k = (taken >> i) & 1u ? 0u : key[i];
        const bool first = k > h.key1, second = k > h.key2;
        h.i2 = first ? h.i1 : second ? i : h.i2;
        h.key2 = first ? h.key1 : second ? k : h.key2;
        h.i1 = first ? i : h.i1;
        h.key1 = first ? k : h.key1;
    }
    return h;
}

// The choice value of a key (not NaN's payload, not 0's sign).
__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// What a group is worth, as a key, from the keys of its best and second best.
__device__ __forceinline__ uint32_t worth_of(uint32_t best, uint32_t second, int group_top)
{
    return group_top == 2 && second > kMaskedKey ? choice_key(value_of(best) + value_of(second)) : best;
}

// Bit g: group g is among the top_groups worthiest.  Groups of whole elements
// of the warp (32, 64, ... experts) are valued by redux; of other sizes by one
// lane each, from shared memory.
template <int V>
__device__ __forceinline__ uint32_t kept_groups(const RouteParams &p, const uint32_t *key, uint32_t *s_key)
{
    const int lane = threadIdx.x & 31, size = p.experts / p.groups;
    uint32_t worth = 0u;   // of group `lane`
    if (size % 32 == 0) {
        const int m = size / 32;
        uint32_t one = 0u, two = 0u;
        int in = 0, g = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            two = max(two, min(one, key[i]));
            one = max(one, key[i]);
            if (++in == m) {
                const uint32_t best = __reduce_max_sync(kFullWarp, one);
                uint32_t second = 0u;
                if (p.group_top == 2) {
                    const uint32_t at = __ballot_sync(kFullWarp, one == best);
                    second = (at & (at - 1u)) ? best   // two lanes have it
                                              : __reduce_max_sync(kFullWarp, one == best ? two : one);
                }
                if (lane == g)
                    worth = worth_of(best, second, p.group_top);
                one = two = 0u;
                in = 0;
                ++g;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (32 * i + lane < p.experts)
                s_key[32 * i + lane] = key[i];
        __syncwarp();
        if (lane < p.groups) {
            uint32_t one = 0u, two = 0u;
            for (int i = 0; i < size; ++i) {
                const uint32_t k = s_key[lane * size + i];
                two = max(two, min(one, k));
                one = max(one, k);
            }
            worth = worth_of(one, two, p.group_top);
        }
        __syncwarp();
    }
    int before = 0;   // groups that go before this one
    for (int g = 0; g < p.groups; ++g) {
        const uint32_t o = __shfl_sync(kFullWarp, worth, g);
        before += (o > worth || (o == worth && g < lane)) ? 1 : 0;
    }
    return __ballot_sync(kFullWarp, lane < p.groups && before < p.top_groups);
}

// Choose and weigh the experts of the tokens first .. last - 1, one after the
// other, by the calling warp; counts each expert's in s_count if there is a plan.
template <int D, int V>
__device__ __forceinline__ void choose_tokens(const RouteParams &p, int64_t first, int64_t last, const float *s_bias,
                                              uint32_t *s_key, uint32_t *s_count)
{
    using T = typename Elem<D>::type;
    const int lane = threadIdx.x & 31;
    const bool by_logit = !p.bias && p.group_top == 1;
    const bool whole = p.softmax && (p.scores || !p.renorm || !by_logit);   // needs the softmax over all experts
    // e / size by a product: exact for e < 512 and sizes up to 256
    const uint32_t inverse = ((1u << 20) + p.experts / p.groups - 1u) / (p.experts / p.groups);
    float x[V];
    const T *row = static_cast<const T *>(p.logits) + first * p.stride;
    auto load_row = [&](const T *from) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = 32 * i + lane < p.experts ? Elem<D>::get(from[32 * i + lane]) : -INFINITY;
    };
    if (first < last)
        load_row(row);
    for (int64_t t = first; t < last; ++t) {
        float top = 0.f, sum = 1.f;
        if (whole) {
            top = x[0];
#pragma unroll
            for (int i = 1; i < V; ++i)
                top = fmaxf(top, x[i]);
            top = value_of(__reduce_max_sync(kFullWarp, top == top ? choice_key(top) : 0u));
            if (!(top > -INFINITY))
                top = 0.f;   // every expert masked (or NaN)
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                sum += expf(x[i] - top);
            sum = warp_sum(sum);
            if (sum == 0.f)
                sum = 1.f;
        }
        uint32_t key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float v = x[i];
            if (!by_logit || p.scores) {
                const float s = p.softmax ? expf(x[i] - top) / sum : sigmoid_of(x[i]);
                if (p.scores && 32 * i + lane < p.experts)
                    p.scores[t * p.experts + 32 * i + lane] = s;
                if (!by_logit) {
                    v = p.bias ? s + s_bias[32 * i + lane] : s;
                    v = x[i] == -INFINITY ? -INFINITY : v;
                }
            }
            key[i] = choice_key(v);
        }
        // the next row is on its way while this one's experts are chosen
        const T *here = row;
        row += p.stride;
        if (t + 1 < last)
            load_row(row);
        if (p.groups > 1) {
            const uint32_t kept = kept_groups<V>(p, key, s_key);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t g = ((32 * i + lane) * inverse) >> 20;   // beyond the groups: already masked
                key[i] = (kept >> (g & 31u)) & 1u ? key[i] : 0u;
            }
        }
        // rounds; lane j keeps place j
        int mine = -1;
        uint32_t taken = 0u;
        Heads h = heads_of<V>(key, 0u);
        for (int j = 0; j < p.top_k; ++j) {
            const uint32_t best = __reduce_max_sync(kFullWarp, h.key1);
            if (best <= kMaskedKey)
                break;
            const uint32_t at = __ballot_sync(kFullWarp, h.key1 == best);
            int e = 32 * h.i1 + lane;
            if (at & (at - 1u)) {   // equals on several lanes: the lowest expert
                e = static_cast<int>(__reduce_min_sync(kFullWarp, h.key1 == best ? static_cast<uint32_t>(e) : ~0u));
            } else {
                e = __shfl_sync(kFullWarp, e, __ffs(at) - 1);
            }
            if (lane == j)
                mine = e;
            if (lane == (e & 31)) {
                taken |= 1u << (e >> 5);
                h.key1 = h.key2;
                h.i1 = h.i2;
                h.key2 = 0u;
            }
            if constexpr (V > 2) {
                // a lane whose second one is gone too has to look again
                const bool empty = h.key1 == 0u && taken != 0u;
                if (__any_sync(kFullWarp, empty && lane == (e & 31)))
                    h = heads_of<V>(key, taken);
            }
        }
        // weights
        const bool there = mine >= 0;
        const float xm = there ? Elem<D>::get(here[mine]) : -INFINITY;
        float w;
        if (p.softmax) {
            if (p.renorm) {
                top = warp_max(xm);
                w = there ? expf(xm - top) : 0.f;
                w = w / warp_sum(w);
            } else {
                w = expf(xm - top) / sum;
            }
        } else {
            w = there ? sigmoid_of(xm) : 0.f;
            if (p.renorm)
                w = w / (warp_sum(w) + 1e-20f);
        }
        if (lane < p.top_k) {
            p.ids[t * p.top_k + lane] = mine;
            p.weights[t * p.top_k + lane] = there ? w * p.scale : 0.f;
        }
        if (p.plan) {
            if (there)
                ++s_count[mine];
            __syncwarp();
        }
    }
}

template <int D, int V>
__global__ void __launch_bounds__(kRouteWarps * 32, 1) route_kernel(const __grid_constant__ RouteParams p)
{
    extern __shared__ uint32_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int E = p.experts;
    const uint32_t cta = blockIdx.x, ctas = gridDim.x;
    uint32_t *s_count = smem;                                          // [warps][E]
    uint32_t *s_base = s_count + (p.plan ? warps * E : 0);             // [E]
    uint32_t *s_sums = s_base + E;                                     // [2][rows at a time][E], up to 4096
    float *s_bias = reinterpret_cast<float *>(s_sums + 4096);          // [32 V]
    uint32_t *s_keys = reinterpret_cast<uint32_t *>(s_bias) + 32 * V;  // [warps][E], groups of odd sizes
    __shared__ uint32_t s_chunk[16];
    __shared__ int s_stop;

    uint32_t tag = 0;
    bool stop = false;
    if (p.plan && warp == 0) {
        tag = ld_relaxed_gpu(p.header + kStepEpochWord) + 1u;
        stop = ld_relaxed_gpu(p.header + kStepStatusWord + 1) != 0u;   // an earlier call failed
    }
    if (p.bias)
        for (int e = threadIdx.x; e < 32 * V; e += blockDim.x)
            s_bias[e] = e < E ? p.bias[e] : -INFINITY;
    if (p.plan)
        for (int i = threadIdx.x; i < warps * E; i += blockDim.x)
            s_count[i] = 0u;
    __syncthreads();

    // the warp's stretch of tokens
    const int64_t begin = p.tokens * cta / ctas, end = p.tokens * (cta + 1) / ctas;
    const int64_t first = begin + (end - begin) * warp / warps, last = begin + (end - begin) * (warp + 1) / warps;
    choose_tokens<D, V>(p, first, last, s_bias, s_keys + warp * E, s_count + warp * E);
    if (!p.plan)
        return;

    // counts of the CTA's warps become the counts before each warp; the CTA's own go to the other CTAs, in
    // 16 bits where no CTA has more tokens than that
    __syncthreads();
    const bool narrow = p.tokens <= static_cast<int64_t>(ctas) * 65535;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        uint32_t run = 0u;
        for (int w = 0; w < warps; ++w) {
            const uint32_t c = s_count[w * E + e];
            s_count[w * E + e] = run;
            run += c;
        }
        s_base[e] = run;
        if (ctas > 1) {
            if (narrow)
                reinterpret_cast<uint16_t *>(p.counts)[cta * (E + (E & 1)) + e] = static_cast<uint16_t>(run);
            else
                p.counts[cta * E + e] = run;
        }
    }
    const int cols = narrow ? (E + 1) / 2 : E, wide = (cols + 31) / 32 * 32;
    const int rows = ctas > 1 ? max(static_cast<int>(blockDim.x) / wide, 1) : 1;   // summed at a time
    uint32_t *s_before = s_sums, *s_total = s_sums + rows * E;
    if (ctas > 1) {
        __syncthreads();
        if (warp == 0) {
            if (!stop) {
                fence_release_gpu();
                send_all(p.header, ctas, tag, 0u);
                uint32_t none[kStepMaxCtas / 32];
                stop = receive_all(p.header, ctas, tag, p.timeout_ns, none);
                fence_acquire_gpu();
                if (!stop && cta == 0 && lane == 0)
                    st_relaxed_gpu(p.header + kStepEpochWord, tag);
            }
            if (lane == 0)
                s_stop = stop;
        }
        __syncthreads();
        if (s_stop)
            return;
        // sum the rows of all CTAs, and of those before this one: some columns and rows a thread
        const int col = threadIdx.x % wide, part = threadIdx.x / wide;
        if (col < cols && part < rows) {
            uint32_t before0 = 0, before1 = 0, total0 = 0, total1 = 0;
#pragma unroll 4
            for (uint32_t r = part; r < ctas; r += rows) {
                const uint32_t c = __ldcg(p.counts + r * cols + col);
                const uint32_t c0 = narrow ? c & 0xffffu : c, c1 = narrow ? c >> 16 : 0u;
                total0 += c0;
                total1 += c1;
                before0 += r < cta ? c0 : 0u;
                before1 += r < cta ? c1 : 0u;
            }
            const int e = narrow ? 2 * col : col;
            s_before[part * E + e] = before0;
            s_total[part * E + e] = total0;
            if (narrow && e + 1 < E) {
                s_before[part * E + e + 1] = before1;
                s_total[part * E + e + 1] = total1;
            }
        }
        __syncthreads();
    } else {
        if (warp == 0 && lane == 0)
            s_stop = stop;
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            s_before[e] = 0u;
            s_total[e] = s_base[e];
        }
        __syncthreads();
        if (s_stop)
            return;
    }
    // where each expert's list starts: a scan over the experts, 32 to a warp
    for (int c = warp; c * 32 < E; c += warps) {
        const int e = c * 32 + lane;
        uint32_t before = 0, total = 0;
        if (e < E) {
            for (int r = 0; r < rows; ++r) {
                before += s_before[r * E + e];
                total += s_total[r * E + e];
            }
        }
        uint32_t run = total;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(kFullWarp, run, d);
            run += lane >= d ? o : 0u;
        }
        if (lane == 31)
            s_chunk[c] = run;
        if (e < E) {
            s_base[e] = run - total + before;
            s_total[e] = run;   // row 0: read only by this lane
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        uint32_t earlier = 0;
        for (int c = 0; c < e / 32; ++c)
            earlier += s_chunk[c];
        s_base[e] += earlier;
        if (cta == 0) {
            if (e == 0)
                p.offsets[0] = 0;
            p.offsets[e + 1] = static_cast<int32_t>(earlier + s_total[e]);
        }
    }
    uint32_t listed = 0;
    for (int c = 0; c * 32 < E; ++c)
        listed += s_chunk[c];
    __syncthreads();

    // phase 2: the same tokens in the same order
    uint32_t *count = s_count + warp * E;
    int id = first < last && lane < p.top_k ? p.ids[first * p.top_k + lane] : -1;
    for (int64_t t = first; t < last; ++t) {
        const int64_t entry = t * p.top_k + lane;
        const int next = t + 1 < last && lane < p.top_k ? p.ids[entry + p.top_k] : -1;
        if (lane < p.top_k) {
            int place = -1;
            if (id >= 0) {
                place = static_cast<int>(s_base[id] + count[id]++);
                p.order[place] = static_cast<int32_t>(entry);
            }
            if (p.places)
                p.places[entry] = place;
        }
        __syncwarp();
        id = next;
    }
    // places that no entry takes
    const int64_t n = p.tokens * p.top_k;
    const int64_t from = max(n * cta / ctas, static_cast<int64_t>(listed));
    for (int64_t i = from + threadIdx.x; i < n * (cta + 1) / ctas; i += blockDim.x)
        p.order[i] = -1;
}

inline size_t route_smem(const RouteParams &p, int V, int warps)
{
    const bool odd_groups = p.groups > 1 && p.experts / p.groups % 32 != 0;
    return sizeof(uint32_t) * ((p.plan ? warps * p.experts : 0) + p.experts + 4096 + 32 * V +
                               (odd_groups ? warps * p.experts : 0));
}

template <int D, int V>
cudaError_t launch_route_v(const RouteParams &p, int ctas, int warps, cudaStream_t s)
{
    const size_t smem = route_smem(p, V, warps);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(route_kernel<D, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess)
            return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute coop;
    coop.id = cudaLaunchAttributeCooperative;
    coop.val.cooperative = 1;
    cfg.attrs = &coop;
    cfg.numAttrs = p.plan && ctas > 1 ? 1 : 0;
    RouteParams arg = p;
    void *args[] = {&arg};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(route_kernel<D, V>), args);
}

// The narrowest kernel that has an element for each expert.
template <int D>
cudaError_t launch_route(const RouteParams &p, int ctas, int warps, cudaStream_t s)
{
    const int v = (p.experts + 31) / 32;
    return v <= 1    ? launch_route_v<D, 1>(p, ctas, warps, s)
           : v <= 2  ? launch_route_v<D, 2>(p, ctas, warps, s)
           : v <= 4  ? launch_route_v<D, 4>(p, ctas, warps, s)
           : v <= 6  ? launch_route_v<D, 6>(p, ctas, warps, s)
           : v <= 8  ? launch_route_v<D, 8>(p, ctas, warps, s)
           : v <= 12 ? launch_route_v<D, 12>(p, ctas, warps, s)
                     : launch_route_v<D, 16>(p, ctas, warps, s);
}

#endif

}  // namespace cns
