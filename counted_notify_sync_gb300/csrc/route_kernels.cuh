// route_kernels.cuh -- the routing kernel: choose each token's experts, weigh
// them, and place the entries by expert.
//
// One warp takes one token: element i of lane l is expert 32 i + l, so every
// load of a row is coalesced whatever its alignment, and among equal choice
// values the lower expert is the lower element, then the lower lane.
//
// Choice.  What a token costs is instructions, not bytes: 1970 of them a token
// of 256 experts, groups and a bias when every choice value was computed
// exactly and carried beside its index (ncu: 66 % of the issue slots, DRAM under
// 1 %).  So the common path works on 32-bit keys, 23 bits of value over the
// expert's number, the lower expert above:
//   - 16-bit logits chosen by logit: their 16 or 19 bits, in order.  Exact.
//   - 32-bit logits chosen by logit: their distance below the row's largest in
//     units of 16 * 2^-23, rounded.  Rounding keeps the order or makes equals.
//   - scores: fixed point over the range that the biases allow, from the
//     hardware's approximate exponential and reciprocal.
// In the last two the chosen values (and the groups') must lie further apart
// than they may be off.  Where they do not (ties; at random one token in some
// hundred) the choice is settled among the few that it is between by their
// exact values; NaN, infinite logits and what is left take the exact path.
// The weights come from the exact scores of the chosen either way.
//   The best eight of a row: each lane keeps its three best keys, the lanes'
// first and second ones go through a sorting network (23 exchanges), and if a
// third one belongs in, or more than eight places are asked for, the places
// are filled in rounds, one redux each.  Four tokens' weights (eight lanes
// each) are computed together.  A bias is part of the offset that a score's
// scaling adds anyway, and keys of one lane carry its number only once they meet
// those of others (not where groups are compared).  Now 530 instructions a token
// of 384 experts with a bias, 76 % of the issue slots and 61 % of the half-rate
// pipe that min, max and compare share (the plan has 70 more): 65536 x 384 bf16
// 48 us, 16384 x 256 f32 with groups 23 us (8.6 and 2.8 us of them are the
// bytes' time).  A softmax's sum, where the weights, the scores or the choice
// need it, is of expf: 3001 x 160 11.6 us, 11.35 by the approximate one.
//
// Plan.  CTA b has a stretch of tokens and each of its warps a stretch of
// those, so that entries in order are warps in order.  The first grid chooses
// and adds its counts per expert to those of its block of 16 CTAs; a second
// grid over the same stretches (route_plan_kernel) counts each warp's ids
// again, sums the blocks and the CTAs of its own block before it, and walks its
// tokens in order, each entry's place being its expert's running count.  Only
// integer sums: the plan does not depend on timing.  The second grid is
// launched early: its CTAs take the places of the first one's as those end, and
// set up while the last ones choose.  (As one cooperative grid with an exchange
// between the phases the plan took as long in a CUDA graph, but 2 us more from
// call to call in a stream, where such a launch cannot be early: 16384 x 256
// 26.1 us against 22.9, 3001 x 160 14.4 against 11.9.)  Of 22.9 us the plan has
// 5: 1.0 until the counts are there, 1.1 to load and count, 1.3 for the scans,
// 1.3 to place.  What needs a 64-bit division is ready before the wait: two of
// them a thread after it were 0.8 us.  A single CTA makes the plan itself.
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
    int64_t tokens;
    int64_t stride;
    int32_t experts, top_k, groups, top_groups, group_top;
    int32_t softmax, renorm, plan;
    float scale;
    uint32_t key_step;   // 512, which the compiler must not know (see choose_tokens)
};

// Launch the kernel for p's choice: by logit or by score (a bias, or groups
// worth two experts), all groups or some.  One translation unit for each type
// and choice (route_*.cu).
cudaError_t launch_route_f32_logit(const RouteParams &p, int ctas, int warps, cudaStream_t s);
cudaError_t launch_route_f32_score(const RouteParams &p, int ctas, int warps, cudaStream_t s);
cudaError_t launch_route_bf16_logit(const RouteParams &p, int ctas, int warps, cudaStream_t s);
cudaError_t launch_route_bf16_score(const RouteParams &p, int ctas, int warps, cudaStream_t s);
cudaError_t launch_route_f16_logit(const RouteParams &p, int ctas, int warps, cudaStream_t s);
cudaError_t launch_route_f16_score(const RouteParams &p, int ctas, int warps, cudaStream_t s);

// Lanes that a token's places take when tokens are handled several at a time.
__device__ __forceinline__ int place_lanes(const RouteParams &p) { return p.top_k <= 8 ? 8 : 32; }

// The tokens of a CTA, and of a warp of it: first .. last - 1.
struct Stretch {
    int64_t first, last;
    __device__ __forceinline__ Stretch(int64_t tokens, int warp, int warps)
    {
        const int64_t begin = tokens * blockIdx.x / gridDim.x, end = tokens * (blockIdx.x + 1) / gridDim.x;
        first = begin + (end - begin) * warp / warps;
        last = begin + (end - begin) * (warp + 1) / warps;
    }
};

// What the CTAs of a plan know of one another: for each expert the count of
// each CTA, in p.counts, and of each block of 16 CTAs, so that nobody has to
// read the counts of all CTAs (152 rows by 152 CTAs took 2.5 us).  The plan
// leaves the blocks' sums cleared.
__device__ __forceinline__ uint32_t *block_sums(const RouteParams &p, uint32_t block)
{
    return p.header + kStepSumWord + block * CNS_ROUTE_MAX_EXPERTS;
}

// The plan, by all threads of a CTA: places the entries of its tokens by
// expert.  s_count: each warp's count of each expert; s_base, s_total: [E].
// held: the ids of the lane's places in the warp's first HELD batches of
// tokens.  before, total: with several CTAs, the entries of earlier ones and
// of all, of expert threadIdx.x.
template <int HELD>
__device__ __forceinline__ void place_entries(const RouteParams &p, const Stretch &mine, const int (&held)[HELD],
                                              uint32_t before, uint32_t total, uint32_t *s_count, uint32_t *s_base,
                                              uint32_t *s_total)
{
    __shared__ uint32_t s_chunk[16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int E = p.experts;
    const uint32_t cta = blockIdx.x, ctas = gridDim.x;
    // One thread an expert: counts of the CTA's warps become the counts before each warp; where the expert's list
    // starts, by a scan over the experts, 32 to a warp.
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        if (e < E) {
            uint32_t run = 0u;
            for (int w = 0; w < warps; w += 8) {
                uint32_t n[8];   // loaded together, before any is stored
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    n[i] = w + i < warps ? s_count[(w + i) * E + e] : 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (w + i < warps)
                        s_count[(w + i) * E + e] = run;
                    run += n[i];
                }
            }
            if (ctas == 1)
                total = run;
        } else {
            total = 0u;
        }
        uint32_t run = total;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(kFullWarp, run, d);
            run += lane >= d ? o : 0u;
        }
        if (lane == 31 && e - lane < E)
            s_chunk[e / 32] = run;
        if (e < E) {
            s_base[e] = run - total + before;
            s_total[e] = run;
        }
    }
    __syncthreads();
    uint32_t listed = 0;
    for (int c = 0; c * 32 < E; ++c)
        listed += s_chunk[c];
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
    __syncthreads();

    // the warp's tokens in order, a batch's entries of one expert ranked by their lanes
    uint32_t *count = s_count + warp * E;
    const int seg = place_lanes(p), per = 32 / seg, place = lane & (seg - 1);
    auto put = [&](int64_t t, int id) {
        const bool token = t < mine.last && place < p.top_k;
        const uint32_t same = __match_any_sync(kFullWarp, id);
        int at = -1;
        if (id >= 0)
            at = static_cast<int>(s_base[id] + count[id] + __popc(same & ((1u << lane) - 1u)));
        __syncwarp();
        if (id >= 0 && (same >> lane) == 1u)   // the last of them
            count[id] += __popc(same);
        __syncwarp();
        if (token) {
            const int64_t entry = t * p.top_k + place;
            if (id >= 0)
                p.order[at] = static_cast<int32_t>(entry);
            if (p.places)
                p.places[entry] = at;
        }
    };
    int64_t t = mine.first + lane / seg;
#pragma unroll
    for (int i = 0; i < HELD; ++i, t += per)
        if (t - lane / seg < mine.last)
            put(t, held[i]);
    for (; t - lane / seg < mine.last; t += per)
        put(t, t < mine.last && place < p.top_k ? p.ids[t * p.top_k + place] : -1);
    // places that no entry takes
    const uint32_t n = static_cast<uint32_t>(p.tokens) * p.top_k;
    for (uint32_t i = listed + cta * blockDim.x + threadIdx.x; i < n; i += ctas * blockDim.x)
        p.order[i] = -1;
}

// Shared memory of place_entries.
inline size_t plan_smem(int experts, int warps) { return sizeof(uint32_t) * (warps + 2) * experts; }

// Let a kernel have `smem` bytes of shared memory; `most` is what any launch of it may ask for, and what it is always
// allowed: another thread's launch may come between this and the caller's, and must not find less.
inline cudaError_t allow_smem(const void *kernel, size_t smem, size_t most)
{
    if (smem <= 48 * 1024)
        return cudaSuccess;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
}

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

// The choice value of a key (not NaN's payload, not 0's sign).
__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// What a group is worth, as a key, from the exact keys of its best and second
// best.
__device__ __forceinline__ uint32_t worth_of(uint32_t best, uint32_t second, int group_top)
{
    return group_top == 2 && second > kMaskedKey ? choice_key(value_of(best) + value_of(second)) : best;
}

// Bit g: group g is among the top_groups worthiest, from exact keys.  Groups of
// whole elements of the warp (32, 64, ... experts) are valued by redux, of other
// sizes by one lane each, from shared memory.
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

// What the fast path's keys are (see the top of the file): a value v becomes
// kQuanta * clamp(v * scale + offset, 0, 1) quanta.
struct KeyRules {
    uint32_t never;   // keys up to this one cannot be chosen
    uint32_t apart;   // quanta between values that are surely in order; 0: keys are exact
    uint32_t zero;    // the quanta of value 0 (scores)
    float scale, offset;
};

constexpr float kNever = -1e30f;   // the value of what cannot be chosen
constexpr float kMostBias = 1e6f;
constexpr float kLeastQuanta = 8388608.f;        // 2^23: a float from there to 2^24 has its integer in its low bits
constexpr float kQuanta = kLeastQuanta - 64.f;

// Scores lie in [0, 1], biases in [1 - reach, reach - 1].  The approximate
// sigmoid's error is s (1 - s) (2^-22 + 2^-23.4 |x|) from the exponential, and
// (2^-24 + 2^-23) s from the sum and the reciprocal: below 2.7e-7.  A softmax
// score's, its sum taken as it is for both ways, is s (2^-22 + 2^-23 |x - top|)
// and two roundings: at the row's largest e^0 is exact and the roundings are
// left, any other's s is at most 1/2 and falls faster than |x - top| grows, so
// it is below 1.8e-7.  What keeps masked experts out adds at most 4.8e-7.  The
// exact score in 32 bits is within 1.8e-7 of the true one: 2.7e-7 + 4.8e-7 +
// 1.8e-7 = 9.3e-7.  The sums with the bias round to 2^-24 of reach each, as the
// near one's offset with the bias in it does.  Two values, and the quanta round
// too.
__device__ __forceinline__ KeyRules score_rules(float reach)
{
    KeyRules r;
    r.never = 511u;
    r.scale = (1.f - 1e-5f) / (2.f * reach - 1.f);
    r.offset = 1e-6f + (reach - 1.f) * r.scale;
    r.zero = static_cast<uint32_t>(r.offset * kQuanta);
    r.apart = 4u + static_cast<uint32_t>(2.f * (9.3e-7f + 1.9e-7f * reach) * r.scale * kQuanta);
    return r;
}

// The row's largest is 0, what lies 16 below it is out of reach.
__device__ __forceinline__ KeyRules logit_rules() { return KeyRules{511u, 1u, 0u, 1.f / 16.f, 1.f}; }

__device__ __forceinline__ KeyRules packed_rules() { return KeyRules{kMaskedKey | 511u, 0u, 0u, 0.f, 0.f}; }

// Whether keys a >= b are surely in this order.
__device__ __forceinline__ bool surely_above(uint32_t a, uint32_t b, uint32_t apart)
{
    return (a >> 9) - (b >> 9) >= apart;
}

// One element's exact choice value as a key; top, sum: of the row's softmax.
__device__ __forceinline__ uint32_t exact_key(const RouteParams &p, float x, float bias, float top, float sum)
{
    float v = x;
    if (p.bias || p.group_top == 2) {
        v = p.softmax ? expf(x - top) / sum : sigmoid_of(x);
        if (p.bias)
            v += bias;
        v = x == -INFINITY ? -INFINITY : v;
    }
    return choice_key(v);
}

// Bit g: group g is among the top_groups worthiest, where the quanta of lane
// g's group's worth leave it open: of those that are neither surely above `most`,
// the best group that is not in, nor surely below `least`, the last that is, by
// their exact worths.
template <int D>
__device__ __noinline__ uint32_t settle_groups(const RouteParams &p, const typename Elem<D>::type *row, uint32_t worth,
                                               uint32_t least, uint32_t most, uint32_t apart, float top, float sum)
{
    const uint32_t lane = threadIdx.x & 31u;
    const int size = p.experts / p.groups;
    const bool group = lane < static_cast<uint32_t>(p.groups), in = group && worth >= most + apart;
    uint32_t kept = __ballot_sync(kFullWarp, in);
    const uint32_t open = __ballot_sync(kFullWarp, group && !in && worth + apart > least);
    uint32_t exact = 0u;   // of lane g's group
    for (uint32_t rest = open; rest; rest &= rest - 1u) {
        const int g = __ffs(rest) - 1;
        uint32_t one = 0u, two = 0u;
        for (int i = lane; i < size; i += 32) {
            const int e = g * size + i;
            const uint32_t k = exact_key(p, Elem<D>::get(row[e]), p.bias ? p.bias[e] : 0.f, top, sum);
            two = max(two, min(one, k));
            one = max(one, k);
        }
        __syncwarp();
        const uint32_t best = __reduce_max_sync(kFullWarp, one), at = __ballot_sync(kFullWarp, one == best);
        const uint32_t second = (at & (at - 1u)) ? best : __reduce_max_sync(kFullWarp, one == best ? two : one);
        exact = lane == static_cast<uint32_t>(g) ? worth_of(best, second, p.group_top) : exact;
    }
    const int places = p.top_groups - __popc(kept);
    int before = 0;
    for (uint32_t rest = open; rest; rest &= rest - 1u) {
        const uint32_t g = __ffs(rest) - 1, o = __shfl_sync(kFullWarp, exact, g);
        before += (o > exact || (o == exact && g < lane)) ? 1 : 0;
    }
    return kept | __ballot_sync(kFullWarp, ((open >> lane) & 1u) && before < places);
}

// The best and the second best over the lanes of each element, to lane i for
// element i < V (a power of two).  Halves of the elements change sides between
// halves of the lanes, so all elements' reductions share the shuffles: 50
// instructions for 8 elements where a redux or two for each took 70 and
// more latency.
template <int V>
__device__ __forceinline__ void best_two_of_each(const uint32_t *key, uint32_t *best, uint32_t *second)
{
    const uint32_t lane = threadIdx.x & 31u;
    uint32_t a[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        a[i] = key[i];
        b[i] = 0u;
    }
    int d = 16;
#pragma unroll
    for (int n = V / 2; n > 0; n >>= 1, d >>= 1) {
        const bool upper = lane & d;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint32_t x = upper ? a[i + n] : a[i], y = __shfl_xor_sync(kFullWarp, upper ? a[i] : a[i + n], d);
            if (n == V / 2) {
                b[i] = min(x, y);
            } else {
                const uint32_t u = upper ? b[i + n] : b[i], w = __shfl_xor_sync(kFullWarp, upper ? b[i] : b[i + n], d);
                b[i] = max(min(x, y), max(u, w));
            }
            a[i] = max(x, y);
        }
    }
    for (; d > 0; d >>= 1) {
        const uint32_t y = __shfl_xor_sync(kFullWarp, a[0], d), w = __shfl_xor_sync(kFullWarp, b[0], d);
        b[0] = max(min(a[0], y), max(b[0], w));
        a[0] = max(a[0], y);
    }
    *best = __shfl_sync(kFullWarp, a[0], (lane * (32 / V)) & 31u);
    *second = __shfl_sync(kFullWarp, b[0], (lane * (32 / V)) & 31u);
}

// Bit g: group g is among the top_groups worthiest, from the fast path's keys,
// which are all different: one redux finds a group's best and a second one,
// without it, the next.
template <int D, int V>
__device__ __forceinline__ uint32_t kept_groups_near(const RouteParams &p, const typename Elem<D>::type *row,
                                                     const uint32_t *key, uint32_t *s_key, int row_groups,
                                                     const KeyRules &rules, float top, float sum)
{
    const uint32_t lane = threadIdx.x & 31u;
    uint32_t best = 0u, second = 0u;   // of group `lane`
    if (V > 1 && (V & (V - 1)) == 0 && row_groups == 1) {
        if constexpr (V > 1 && (V & (V - 1)) == 0)
            best_two_of_each<V>(key, &best, &second);
    } else if (row_groups == 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t top = __reduce_max_sync(kFullWarp, key[i]);
            best = lane == i ? top : best;
            if (p.group_top == 2) {
                const uint32_t next = __reduce_max_sync(kFullWarp, key[i] == top ? 0u : key[i]);
                second = lane == i ? next : second;
            }
        }
    } else {
        // some lanes a group, from shared memory
        const int size = p.experts / p.groups;
        const int lanes = p.groups > 16 ? 1 : p.groups > 8 ? 2 : p.groups > 4 ? 4 : 8;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (32 * i + static_cast<int>(lane) < p.experts)
                s_key[32 * i + lane] = key[i];
        __syncwarp();
        const int g = lane / lanes;
        if (g < p.groups) {
            const uint32_t *mine = s_key + g * size;
#pragma unroll 4
            for (int i = lane & (lanes - 1); i < size; i += lanes) {
                second = max(second, min(best, mine[i]));
                best = max(best, mine[i]);
            }
        }
        for (int d = 1; d < lanes; d <<= 1) {
            const uint32_t b = __shfl_xor_sync(kFullWarp, best, d), c = __shfl_xor_sync(kFullWarp, second, d);
            second = max(min(best, b), max(second, c));
            best = max(best, b);
        }
        // group g's from its first lane to lane g
        best = __shfl_sync(kFullWarp, best, (lane * lanes) & 31);
        second = __shfl_sync(kFullWarp, second, (lane * lanes) & 31);
        __syncwarp();
    }
    uint32_t worth = best;
    if (p.group_top == 2) {   // in quanta, of two values; a masked one adds nothing
        const uint32_t sum = best <= rules.never ? 0u : (best >> 9) + (second <= rules.never ? rules.zero : second >> 9);
        worth = sum << 5 | (31u - lane);
    }
    if (lane >= static_cast<uint32_t>(p.groups))
        worth = 0u;
    // the worthiest, one after the other, and the one after them
    const uint32_t its = worth;
    uint32_t kept = 0u, least = 0u;
    for (int j = 0; j < p.top_groups; ++j) {
        least = __reduce_max_sync(kFullWarp, worth);
        kept |= __ballot_sync(kFullWarp, worth == least);
        worth = worth == least ? 0u : worth;
    }
    if (rules.apart) {
        const uint32_t most = __reduce_max_sync(kFullWarp, worth);
        const int shift = p.group_top == 2 ? 5 : 9;
        const uint32_t apart = p.group_top == 2 ? 2u * rules.apart : rules.apart;
        if ((least >> shift) - (most >> shift) < apart)
            kept = settle_groups<D>(p, row, its >> shift, least >> shift, most >> shift, apart, top, sum);
    }
    return kept;
}

// One exchange of a sorting network: the larger value goes to the lanes that
// have `larger`.
__device__ __forceinline__ uint32_t exchange(uint32_t v, int distance, bool larger)
{
    const uint32_t o = __shfl_xor_sync(kFullWarp, v, distance);
    return larger ? max(v, o) : min(v, o);
}

// Sort the bitonic eights of the warp (lanes 0-7, 8-15, ...), falling where `fall`.
__device__ __forceinline__ uint32_t merge_eights(uint32_t v, bool fall)
{
    const uint32_t lane = threadIdx.x & 31u;
#pragma unroll
    for (int d = 4; d > 0; d >>= 1)
        v = exchange(v, d, ((lane & d) == 0) == fall);
    return v;
}

// Sort the eights of the warp.
__device__ __forceinline__ uint32_t sort_eights(uint32_t v, bool fall)
{
    const uint32_t lane = threadIdx.x & 31u;
    v = exchange(v, 1, ((lane & 1) == 0) == ((lane & 2) == 0));
    v = exchange(v, 2, ((lane & 2) == 0) == ((lane & 4) == 0));
    v = exchange(v, 1, ((lane & 1) == 0) == ((lane & 4) == 0));
    return merge_eights(v, fall);
}

// The eight largest of the lanes' `one` and `two`, falling, in each eight of
// the warp; *rest: the largest of the others.
__device__ __forceinline__ uint32_t best_eight(uint32_t one, uint32_t two, uint32_t *rest)
{
    const uint32_t lane = threadIdx.x & 31u;
    one = sort_eights(one, true);
    two = sort_eights(two, false);
    uint32_t v = max(one, two), other = min(one, two);   // falling against rising: the eight larger, bitonic
    v = merge_eights(v, (lane & 8) == 0);
    uint32_t o = __shfl_xor_sync(kFullWarp, v, 8);
    other = max(other, min(v, o));
    v = merge_eights(max(v, o), (lane & 16) == 0);
    o = __shfl_xor_sync(kFullWarp, v, 16);
    other = max(other, min(v, o));
    *rest = other;
    return merge_eights(max(v, o), true);
}

// The exact path: lane j gets place j's expert (-1: none).
template <int D, int V>
__device__ __noinline__ int choose_exact(const RouteParams &p, const typename Elem<D>::type *row, uint32_t *s_key,
                                         float top, float sum)
{
    const int lane = threadIdx.x & 31;
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = 32 * i + lane;
        key[i] = e < p.experts ? exact_key(p, Elem<D>::get(row[e]), p.bias ? p.bias[e] : 0.f, top, sum) : 0u;
    }
    if (p.groups > p.top_groups) {
        const int size = p.experts / p.groups;
        const uint32_t kept = kept_groups<V>(p, key, s_key);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (32 * i + lane < p.experts && !((kept >> ((32 * i + lane) / size)) & 1u))
                key[i] = 0u;
    }
    int mine = -1;
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t best = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i)
            best = max(best, key[i]);
        best = __reduce_max_sync(kFullWarp, best);
        if (best <= kMaskedKey)
            break;
        uint32_t e = ~0u;   // the lowest expert that has it
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            e = key[i] == best ? 32u * i + lane : e;
        e = __reduce_min_sync(kFullWarp, e);
        if (lane == j)
            mine = static_cast<int>(e);
#pragma unroll
        for (int i = 0; i < V; ++i)
            key[i] = 32u * i + lane == e ? 0u : key[i];
    }
    return mine;
}

// Settles a token whose near keys leave its choice open: the experts whose keys
// are not surely below the last place's, at most 32 (false if there are more),
// in the order of their exact choice values, the lower first among equals.
// Lane `place` of each `seg` lanes gets place `place`'s.
template <int D, int V>
__device__ __noinline__ bool settle(const RouteParams &p, const typename Elem<D>::type *row, const uint32_t *key,
                                    uint32_t last, uint32_t apart, uint16_t *s_near, int seg, float top, float sum,
                                    int *chosen)
{
    const uint32_t lane = threadIdx.x & 31u, earlier = (1u << lane) - 1u;
    const uint32_t quanta = last >> 9;
    const uint32_t least = max((quanta > apart ? quanta - apart : 0u) << 9, 511u);   // 511: nothing that is no expert
    uint32_t count = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const bool in = key[i] > least;
        const uint32_t at = __ballot_sync(kFullWarp, in), to = count + __popc(at & earlier);
        if (in && to < 32u)
            s_near[to] = static_cast<uint16_t>(32 * i + lane);
        count += __popc(at);
    }
    if (count > 32u)
        return false;
    __syncwarp();
    const int e = lane < count ? s_near[lane] : -1;
    const uint32_t exact = e >= 0 ? exact_key(p, Elem<D>::get(row[e]), p.bias ? p.bias[e] : 0.f, top, sum) : 0u;
    uint32_t before = 0u;
    for (uint32_t j = 0; j < count; ++j) {
        const uint32_t k = __shfl_sync(kFullWarp, exact, j);
        const int o = __shfl_sync(kFullWarp, e, j);
        before += (k > exact || (k == exact && o < e)) ? 1u : 0u;
    }
    __syncwarp();
    if (e >= 0)
        s_near[before] = static_cast<uint16_t>(e);
    __syncwarp();
    const int place = lane & (seg - 1);
    *chosen = place < p.top_k ? s_near[place] : -1;
    __syncwarp();
    return true;
}

// The sum, or the largest, over the calling lane's `seg` lanes.
__device__ __forceinline__ float seg_sum(float v, int seg)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        if (d < seg)
            v += __shfl_xor_sync(kFullWarp, v, d);
    return v;
}

__device__ __forceinline__ float seg_max(float v, int seg)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        if (d < seg)
            v = fmaxf(v, __shfl_xor_sync(kFullWarp, v, d));
    return v;
}

// Whether a token's keys go through shared memory, for groups that are not one row of 32 experts.
__host__ __device__ __forceinline__ bool odd_groups(const RouteParams &p)
{
    return p.groups > 1 && p.experts / p.groups != 32;
}

// Rows of 32 experts that the next narrower kernel has (launch_route).
__host__ __device__ constexpr int narrower(int v)
{
    return v > 12 ? 12 : v > 8 ? 8 : v > 6 ? 6 : v > 4 ? 4 : v > 2 ? 2 : v - 1;
}

// Choose and weigh the experts of the tokens first .. last - 1 by the calling
// warp; counts each expert's in s_count if there is a plan.  s_offset: what the
// scaled score of expert e is added to, kNever where the bias is -inf and beyond
// the last expert; reach: 1 plus the largest magnitude among the other biases,
// or NaN if they are nothing that the fast path is made for.
// Returns the last batch's expert of the lane's place: of all tokens, if they
// are one batch.
template <int D, int V, bool SCORES, bool GROUPS>
__device__ __forceinline__ int choose_tokens(const RouteParams &p, int64_t first, int64_t last, const float *s_offset,
                                              float reach, uint32_t *s_key, uint16_t *s_near, uint32_t *s_count)
{
    using T = typename Elem<D>::type;
    const int lane = threadIdx.x & 31;
    constexpr bool by_logit = !SCORES;
    const bool whole = p.softmax && (p.scores || !p.renorm || !by_logit);   // needs the softmax over all experts
    constexpr bool packs = D != CNS_DT_F32 && by_logit;
    // keys of a lane need not say which lane's they are until they meet other lanes'
    constexpr bool lanes_later = !packs && !GROUPS;
    const KeyRules rules = packs ? packed_rules() : by_logit ? logit_rules() : score_rules(reach);
    // e / size by a product: exact for e < 512 and sizes up to 256
    const int size = p.experts / p.groups;
    const uint32_t inverse = ((1u << 20) + size - 1u) / size;
    const int row_groups = size % 32 == 0 ? size / 32 : 0;   // rows of 32 experts in a group
    const int seg = place_lanes(p), per = 32 / seg;
    const int place = lane & (seg - 1);
    const T *row = static_cast<const T *>(p.logits) + first * p.stride;
    int held = 0;                // tokens of the batch
    int mine = -1, done = -1;    // of the lane's token, its place's expert
    float its_top = 0.f, its_sum = 1.f;
    for (int64_t t = first; t < last; ++t, row += p.stride) {
        // the next row is on its way to L1 while this one's experts are chosen
        if (t + 1 < last && lane < V)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(row + p.stride + min(32 * lane, p.experts - 1)));
        uint32_t key[V];
        bool sure = by_logit || reach == reach;
        bool none = false;
        float top = 0.f, sum = 1.f;
        {
            float x[V];
#pragma unroll
            for (int i = 0; i < V; ++i)   // (rows that the next narrower kernel has are whole)
                x[i] = i < narrower(V) || 32 * i + lane < p.experts ? Elem<D>::get(row[32 * i + lane]) : -INFINITY;
            if (whole || (by_logit && !packs)) {
                top = x[0];
#pragma unroll
                for (int i = 1; i < V; ++i)
                    top = fmaxf(top, x[i]);
                top = value_of(__reduce_max_sync(kFullWarp, top == top ? choice_key(top) : 0u));
                if (!(top > -INFINITY))
                    top = 0.f;   // every expert masked (or NaN)
            }
            if (whole) {
                sum = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    sum += expf(x[i] - top);
                sum = warp_sum(sum);
                if (sum == 0.f)
                    sum = 1.f;
            }
            if (p.scores) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (32 * i + lane < p.experts)
                        p.scores[t * p.experts + 32 * i + lane] =
                            p.softmax ? expf(x[i] - top) / sum : sigmoid_of(x[i]);
            }
            if (packs) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    key[i] = (choice_key(x[i]) & ~511u) | (511u - (32 * i + lane));
            } else {
                // The arithmetic stays on the FMA pipe where it can: min, max, compare and select go at half its
                // rate, and the keys' comparisons below are many of them.  So the clamp is a saturating product,
                // and the shift a product by a number that the compiler cannot turn into one.
                float all = 0.f, some = 0.f;   // NaN or inf if any value is; 0 if every expert is masked
                auto take = [&](int i, float v, float offset) {
                    all += v;
                    float part;
                    asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(part) : "f"(v), "f"(rules.scale), "f"(offset));
                    if (GROUPS)
                        some += part;
                    key[i] = __float_as_uint(fmaf(part, kQuanta, kLeastQuanta)) * p.key_step +
                             (lanes_later ? 480u - 32u * i : 511u - 32u * i - lane);
                };
                // a score; the least float times the logit is -inf for a masked expert, else below 4.8e-7
                auto take_score = [&](int i, float s) { take(i, fmaf(x[i], 1.4e-45f, s), s_offset[32 * i + lane]); };
                if (by_logit) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        take(i, x[i] - top, rules.offset);
                } else if (p.softmax) {
                    const float inverse = 1.f / sum;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        take_score(i, exp_near(x[i] - top) * inverse);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float s;
                        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + exp_near(-x[i])));
                        take_score(i, s);
                    }
                }
                sure = sure && !__any_sync(kFullWarp, !(all < INFINITY));
                none = GROUPS && __all_sync(kFullWarp, some == 0.f);   // a padded token
            }
        }
        if (GROUPS && sure && !none) {
            const uint32_t kept = kept_groups_near<D, V>(p, row, key, s_key, row_groups, rules, top, sum);
            if (row_groups) {
                uint32_t bits = kept;
                int in = 0;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    key[i] = bits & 1u ? key[i] : 0u;
                    if (++in == row_groups) {
                        bits >>= 1;
                        in = 0;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t g = ((32 * i + lane) * inverse) >> 20;   // beyond the groups: never chosen
                    key[i] = (kept >> (g & 31u)) & 1u ? key[i] : 0u;
                }
            }
        }
        int chosen = -1;   // of place `place`
        if (sure && !none) {
            uint32_t one = 0u, two = 0u, three = 0u;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t k = key[i], a = min(one, k), b = min(two, a);
                one = max(one, k);
                two = max(two, a);
                three = max(three, b);
            }
            if (lanes_later) {
                none = __all_sync(kFullWarp, one <= rules.never);
                one += 31u - lane;
                two += 31u - lane;
                three += 31u - lane;
            }
            // the best key that place `place` can have, and the best one after the last place
            uint32_t got, after = 0u;
            bool rounds = seg != 8;
            if (!rounds) {
                uint32_t rest;
                got = best_eight(one, two, &rest);
                const uint32_t third = V > 2 ? __reduce_max_sync(kFullWarp, three) : 0u;
                const uint32_t last_one = __shfl_sync(kFullWarp, got, p.top_k - 1);
                rounds = V > 2 && third > last_one;   // it belongs in
                if (rules.apart)
                    after = max(max(third, __reduce_max_sync(kFullWarp, rest)),
                                p.top_k < 8 ? __shfl_sync(kFullWarp, got, p.top_k & 7) : 0u);
            }
            if (rounds) {
                got = 0u;
                for (int j = 0; j < p.top_k; ++j) {
                    const uint32_t best = __reduce_max_sync(kFullWarp, one);
                    if (best <= rules.never)
                        break;
                    got = place == j ? best : got;
                    const bool owner = one == best;
                    if (owner) {
                        one = two;
                        two = 0u;
                    }
                    if (V > 2 && __any_sync(kFullWarp, owner && one == 0u)) {
                        // its second one is gone too: look again, below what it gave
                        if (owner) {
#pragma unroll
                            for (int i = 0; i < V; ++i) {
                                const uint32_t whole_key = key[i] + (lanes_later ? 31u - lane : 0u);
                                const uint32_t k = whole_key < best ? whole_key : 0u;
                                two = max(two, min(one, k));
                                one = max(one, k);
                            }
                        }
                        __syncwarp();
                    }
                }
                after = __reduce_max_sync(kFullWarp, one);
            }
            chosen = place < p.top_k && got > rules.never ? static_cast<int>(511u - (got & 511u)) : -1;
            if (rules.apart) {
                // nothing but experts, and nothing that ranks by less than it may be off
                const uint32_t down = __shfl_down_sync(kFullWarp, got, 1);
                const uint32_t next = place + 1 < p.top_k ? down : after;
                sure = none || !__any_sync(kFullWarp, place < p.top_k && chosen < 0);
                if (sure && !none && __any_sync(kFullWarp, place < p.top_k && !surely_above(got, next, rules.apart)))
                    sure = settle<D, V>(p, row, key, __shfl_sync(kFullWarp, got, p.top_k - 1), rules.apart, s_near, seg,
                                        top, sum, &chosen);
            }
        }
        if (!sure) {
            chosen = choose_exact<D, V>(p, row, s_key, top, sum);
            chosen = __shfl_sync(kFullWarp, chosen, place);
        }
        // the lanes of the token's turn take it over
        const bool turn = seg == 32 || (lane >> 3) == held;
        mine = turn ? chosen : mine;
        its_top = turn ? top : its_top;
        its_sum = turn ? sum : its_sum;
        if (++held < per && t + 1 < last)
            continue;
        // weights of the batch
        const int64_t its = t + 1 - held + lane / seg;   // the lane's token
        const bool token = lane / seg < held && place < p.top_k, there = token && mine >= 0;
        const float xm =
            there ? Elem<D>::get(static_cast<const T *>(p.logits)[its * p.stride + mine]) : -INFINITY;
        float w;
        if (p.softmax) {
            if (p.renorm) {
                const float best = seg_max(xm, seg);
                w = there ? expf(xm - best) : 0.f;
                w = w / seg_sum(w, seg);
            } else {
                w = expf(xm - its_top) / its_sum;
            }
        } else {
            w = there ? sigmoid_of(xm) : 0.f;
            if (p.renorm)
                w = w / (seg_sum(w, seg) + 1e-20f);
        }
        if (token) {
            p.ids[its * p.top_k + place] = mine;
            p.weights[its * p.top_k + place] = there ? w * p.scale : 0.f;
        }
        if (p.plan && there)
            atomicAdd(&s_count[mine], 1u);
        held = 0;
        done = token ? mine : -1;
        mine = -1;
    }
    return done;
}

// Chooses, and counts if there is a plan; a single CTA makes the plan too.
template <int D, int V, bool SCORES, bool GROUPS>
__global__ void __launch_bounds__(kRouteWarps * 32, 1) route_kernel(const __grid_constant__ RouteParams p)
{
    extern __shared__ uint32_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int E = p.experts;
    const uint32_t cta = blockIdx.x, ctas = gridDim.x;
    const bool alone = ctas == 1;
    float *s_offset = reinterpret_cast<float *>(smem);                     // [32 V]
    uint32_t *s_keys = smem + 32 * V;                                      // [warps][E], groups of other sizes than 32
    uint32_t *s_count = s_keys + (odd_groups(p) ? warps * E : 0);          // [E], or for a single CTA [warps][E]
    __shared__ int s_stop, s_reach;
    __shared__ uint16_t s_near[kRouteWarps][32];   // experts that a token's choice is between

    const Stretch mine(p.tokens, warp, warps);
    if (threadIdx.x == 0)
        s_reach = 0;
    if (p.plan)
        for (int i = threadIdx.x; i < (alone ? warps * E : E); i += blockDim.x)
            s_count[i] = 0u;
    grid_dependency_wait();   // launched early: nothing of the tensors or the workspace before this
    if (p.plan && !alone)
        grid_launch_dependents();   // the plan's CTAs take the places of this grid's as those end
    // the warp's first row and the biases are on their way while the CTA sets up
    if (mine.first < mine.last && lane < V) {
        const int e = min(lane * 32, E - 1);
        asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const typename Elem<D>::type *>(p.logits) +
                                                      mine.first * p.stride + e));
    }
    float b = p.bias && static_cast<int>(threadIdx.x) < E ? p.bias[threadIdx.x] : 0.f;
    __syncthreads();
    if (SCORES) {
        for (int e = threadIdx.x; e < 32 * V; e += blockDim.x) {
            if (e >= static_cast<int>(blockDim.x))
                b = p.bias && e < E ? p.bias[e] : 0.f;
            const bool never = e >= E || b == -INFINITY;
            s_offset[e] = never ? kNever : b;
            // magnitudes compare as integers, NaN above all
            const uint32_t most = __reduce_max_sync(kFullWarp, never ? 0u : __float_as_uint(fabsf(b)));
            if (lane == 0 && most)
                atomicMax(&s_reach, static_cast<int>(most));
        }
        __syncthreads();
    }
    float reach = 1.f + __int_as_float(s_reach);
    reach = reach <= kMostBias ? reach : NAN;
    if (SCORES) {
        const KeyRules rules = score_rules(reach);
        for (int e = threadIdx.x; e < 32 * V; e += blockDim.x)
            s_offset[e] = s_offset[e] == kNever ? kNever : fmaf(s_offset[e], rules.scale, rules.offset);
        __syncthreads();
    }

    const int done = choose_tokens<D, V, SCORES, GROUPS>(p, mine.first, mine.last, s_offset, reach, s_keys + warp * E,
                                                         s_near[warp], s_count + (alone ? warp * E : 0));
    if (!p.plan)
        return;
    if (threadIdx.x == 0)   // read by one thread of a CTA: all threads' loads of one line took 2 us
        s_stop = alone && ld_relaxed_gpu(p.header + kStepStatusWord + 1) != 0u;   // an earlier call failed
    __syncthreads();
    if (alone) {
        const int held[1] = {done};   // a warp of a single CTA has a token at most, or a batch of them
        if (!s_stop)
            place_entries(p, mine, held, 0u, 0u, s_count, s_count + warps * E, s_count + (warps + 1) * E);
        return;
    }
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        const uint32_t n = s_count[e];
        p.counts[cta * E + e] = n;
        if (n)
            red_add_relaxed_gpu(block_sums(p, cta / kStepBlockCtas) + e, n);
    }
}

inline size_t route_smem(const RouteParams &p, int V, int ctas, int warps)
{
    return sizeof(uint32_t) * (32 * V + (odd_groups(p) ? warps * p.experts : 0) + (p.plan && ctas > 1 ? p.experts : 0)) +
           (p.plan && ctas == 1 ? plan_smem(p.experts, warps) : 0);
}

// The largest route_smem of a kernel: 32 V experts in odd groups, and a single CTA's plan.
constexpr size_t most_route_smem(int V)
{
    return sizeof(uint32_t) * 32 * V * (1 + kRouteWarps + kRouteWarps + 2);
}

template <int D, int V, bool SCORES, bool GROUPS>
cudaError_t launch_route_v(const RouteParams &p, int ctas, int warps, cudaStream_t s)
{
    const auto kernel = route_kernel<D, V, SCORES, GROUPS>;
    const size_t smem = route_smem(p, V, ctas, warps);
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), smem, most_route_smem(V));
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = early_launch(&attr);
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    RouteParams arg = p;
    void *args[] = {&arg};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(kernel), args);
}

// The narrowest kernel that has an element for each expert.
template <int D, bool SCORES, bool GROUPS>
cudaError_t launch_route(const RouteParams &p, int ctas, int warps, cudaStream_t s)
{
    const int v = (p.experts + 31) / 32;
    return v <= 1    ? launch_route_v<D, 1, SCORES, GROUPS>(p, ctas, warps, s)
           : v <= 2  ? launch_route_v<D, 2, SCORES, GROUPS>(p, ctas, warps, s)
           : v <= 4  ? launch_route_v<D, 4, SCORES, GROUPS>(p, ctas, warps, s)
           : v <= 6  ? launch_route_v<D, 6, SCORES, GROUPS>(p, ctas, warps, s)
           : v <= 8  ? launch_route_v<D, 8, SCORES, GROUPS>(p, ctas, warps, s)
           : v <= 12 ? launch_route_v<D, 12, SCORES, GROUPS>(p, ctas, warps, s)
                     : launch_route_v<D, 16, SCORES, GROUPS>(p, ctas, warps, s);
}

#endif

}  // namespace cns
