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
// own bytes and no sum needs an atomic.  At most one product and one sum a
// byte or two: HBM bounds them, and a launch the small ones (8 tokens of 4096
// bf16, 8 places: 1.7 us as a kernel of a CUDA graph, 2.3 combined).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "cns.h"
#include "cns_host.h"
#include "rows_device.cuh"

namespace cns {
namespace {

// How a CTA's threads lie over tokens and a row's accesses.
//   Accesses of 16 bytes, one a thread: a CTA has `per` groups of `lanes` threads, each for tokens of its own, or (per =
// 1) one of `parts` stretches of a row.
//   Narrower ones (rows at odd addresses), several a thread, 16 bytes in all, so that it has more than one element's
// work: a warp (lanes = 32, per = 8) has one of `parts` stretches of a row, its lanes neighbouring accesses each time.
struct Tiling {
    uint32_t units, lanes, per, parts, threads, ctas;
};

constexpr uint32_t kRowThreads = 256;

// Accesses of A bytes that a thread holds of a row.
__host__ __device__ constexpr int accesses(int a) { return a == 1 ? 8 : 16 / a; }

// `tokens`: of a thread.
bool tile(int64_t count, int64_t units, int access, uint32_t tokens, Tiling *t)
{
    t->units = static_cast<uint32_t>(units);
    int64_t ctas;
    if (access == 16) {
        t->parts = (t->units + kRowThreads - 1) / kRowThreads;
        t->lanes = (t->units + t->parts - 1) / t->parts;
        t->per = std::max<uint32_t>(1u, kRowThreads / t->lanes);
        t->threads = (t->per * t->lanes + 31) / 32 * 32;
        const int64_t each = static_cast<int64_t>(t->per) * tokens;
        ctas = (count + each - 1) / each * t->parts;
    } else {
        t->lanes = 32;
        t->per = kRowThreads / 32;
        t->parts = (t->units + 32 * accesses(access) - 1) / (32 * accesses(access));
        t->threads = kRowThreads;
        ctas = ((count + tokens - 1) / tokens * t->parts + t->per - 1) / t->per;
    }
    t->ctas = static_cast<uint32_t>(ctas);
    return ctas <= (1 << 29);   // warps are counted in 32 bits; more of them than that no memory has rows for
}

// The first token of the calling thread (the others follow) and its first access (the others are 32 apart each).
template <int A, int TOKENS>
__device__ __forceinline__ void my_place(const Tiling &m, uint32_t cta, int64_t *t, uint32_t *u)
{
    if constexpr (A < 16) {
        const uint32_t warp = cta * (kRowThreads / 32) + threadIdx.x / 32, block = warp / m.parts;
        *t = static_cast<int64_t>(block) * TOKENS;
        *u = (warp - block * m.parts) * (32 * accesses(A)) + threadIdx.x % 32;
    } else {
        uint32_t group = 0, block = cta, part = 0;
        if (m.parts == 1) {
            group = threadIdx.x / m.lanes;
        } else {
            block = cta / m.parts;
            part = cta % m.parts;
        }
        const uint32_t lane = threadIdx.x - group * m.lanes;
        *t = (static_cast<int64_t>(block) * m.per + group) * TOKENS;
        *u = group < m.per && lane < m.lanes ? part * m.lanes + lane : m.units;
    }
}

struct DispatchParams {
    const uint8_t *x;
    uint8_t *rows;
    const uint8_t *scales;
    uint8_t *row_scales;
    const int32_t *places;
    int64_t tokens, x_stride, scales_stride;
    uint32_t rows_stride, row_scales_stride;   // below 2^32, so that a row's offset is one product
    uint32_t limit;                            // rows
    int32_t top_k, scale_access;
    Tiling data, scale;
};

// A token's accesses are read once and stored top_k times; the loads are a small part, so many small CTAs keep enough
// stores on their way.  16384 x 4096 e4m3 and 32 scales, 8 places: 92.8 us, 99 % of its bytes at the copy rate; bf16
// 177.8 us, 100 %; 8192 x 2049 bf16 (odd rows, accesses of 2 bytes), 4 places: 33.5 us, 74 %.
template <int A>
__device__ __forceinline__ void move(const DispatchParams &p, const Tiling &m, uint32_t cta, const uint8_t *from,
                                     int64_t from_stride, uint8_t *to, uint32_t to_stride)
{
    using B = typename Bits<A>::type;
    constexpr int H = accesses(A);
    int64_t t;
    uint32_t u;
    my_place<A, 1>(m, cta, &t, &u);
    if (u >= m.units || t >= p.tokens)
        return;
    const B *x = reinterpret_cast<const B *>(from + t * from_stride) + u;
    const int32_t *place = p.places + t * p.top_k;
    const auto go = [&](auto full) {   // whether all its accesses are within the row
        const auto within = [&](int h) { return decltype(full)::value || u + 32 * h < m.units; };
        B v[H];
#pragma unroll
        for (int h = 0; h < H; ++h)
            if (within(h))
                v[h] = x[32 * h];
#pragma unroll 4
        for (int j = 0; j < p.top_k; ++j) {
            const uint32_t row = static_cast<uint32_t>(place[j]);
            if (row < p.limit) {
                B *y = reinterpret_cast<B *>(to + static_cast<uint64_t>(row) * to_stride) + u;
#pragma unroll
                for (int h = 0; h < H; ++h)
                    if (within(h))
                        y[32 * h] = v[h];
            }
        }
    };
    if (A == 16 || u - threadIdx.x % 32 + 32 * H <= m.units)
        go(std::true_type());
    else
        go(std::false_type());
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
    int64_t tokens, base_stride, y_stride;   // elements
    int64_t step;                            // a thread's tokens from one round to the next
    uint32_t rows_stride;                    // elements, below 2^30
    uint32_t limit;
    int32_t top_k;
    Tiling data;
};

// CTAs to an SM that combine's registers are shared out for, by the rows that a thread has in flight: 64 registers a
// thread where those are up to four, else 80.  (Two places of two tokens in bf16 put 48 bytes a thread aside for that, one
// place of two in f16 eight; the others fit.)  Narrow accesses have three CTAs (four spill).
__host__ __device__ constexpr int combine_ctas(int a, int rows) { return a == 16 && rows <= 4 ? 4 : 3; }

// What a thread of combine_kernel does; FULL: all its accesses are within the row.
template <int D, int A, int BATCH, int TOKENS, bool FULL>
__device__ __forceinline__ void combine_rows(const CombineParams &p, int64_t t, uint32_t u)
{
    using T = typename Elem<D>::type;
    using B = typename Bits<A>::type;
    constexpr int V = A / static_cast<int>(sizeof(T)), H = accesses(A);
    const auto within = [&](int h) { return FULL || u + 32 * h < p.data.units; };
    const T *rows = static_cast<const T *>(p.rows) + static_cast<int64_t>(u) * V;
    uint32_t next[TOKENS][BATCH];
    const auto places = [&](int64_t of, int j) {
#pragma unroll
        for (int n = 0; n < TOKENS; ++n)
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                next[n][i] = 0xffffffffu;
                if (of + n < p.tokens && j + i < p.top_k)
                    next[n][i] = static_cast<uint32_t>(p.places[(of + n) * p.top_k + j + i]);
            }
    };
    places(t, 0);
    float sum[TOKENS][H][V] = {};
    int j = 0;
    while (t < p.tokens) {
        bool there[TOKENS][BATCH];
        B raw[TOKENS][BATCH][H];
#pragma unroll
        for (int n = 0; n < TOKENS; ++n)
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                there[n][i] = next[n][i] < p.limit;
                const B *row = reinterpret_cast<const B *>(rows + static_cast<uint64_t>(next[n][i]) * p.rows_stride);
#pragma unroll
                for (int h = 0; h < H; ++h)
                    raw[n][i][h] = B{};
                if (there[n][i]) {
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        if (within(h))
                            raw[n][i][h] = row[32 * h];
                }
            }
        const int64_t now = t;
        const int place = j;
        j += BATCH;
        if (j >= p.top_k) {
            j = 0;
            t += p.step;
        }
        places(t, j);
#pragma unroll
        for (int n = 0; n < TOKENS; ++n)
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                // what is not there: 0 * 0
                const float weight = !there[n][i] ? 0.f : p.weights ? p.weights[(now + n) * p.top_k + place + i] : 1.f;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    float v[V];
                    unpack<D, A>(raw[n][i][h], v);
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        sum[n][h][k] = fmaf(weight, v[k], sum[n][h][k]);
                }
            }
        if (j != 0)
            continue;
#pragma unroll
        for (int n = 0; n < TOKENS; ++n) {
            if (now + n >= p.tokens)
                break;
            const B *base = reinterpret_cast<const B *>(static_cast<const T *>(p.base) + (now + n) * p.base_stride) + u;
            B *y = reinterpret_cast<B *>(static_cast<T *>(p.y) + (now + n) * p.y_stride) + u;
            if (p.base) {
                B raw_base[H];
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    raw_base[h] = B{};
                    if (within(h))
                        raw_base[h] = base[32 * h];
                }
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    float v[V];
                    unpack<D, A>(raw_base[h], v);
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        sum[n][h][k] += v[k];
                }
            }
#pragma unroll
            for (int h = 0; h < H; ++h)
                if (within(h))
                    y[32 * h] = pack<D, A>(sum[n][h]);
        }
#pragma unroll
        for (int n = 0; n < TOKENS; ++n)
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    sum[n][h][k] = 0.f;
    }
}

// A thread has TOKENS tokens at a time and of each the rows of BATCH places, all in flight together; while they are on
// their way it loads the places of the next ones.  As many CTAs as the GPU holds, so that only a thread's first rows wait
// for their places: 65536 x 1024 bf16 with two places takes 66.9 us, 89 % of the copy rate; a CTA for every 256 accesses,
// each waiting for its places, took 91.  16384 x 4096 bf16, 8 places: 179 us as a dispatch's gradient (99 %), 201 with
// weights and a base (98 %).  8192 x 2049 bf16, 4 places: 47.1 us (53 %; instructions).
template <int D, int A, int BATCH, int TOKENS>
__global__ void __launch_bounds__(kRowThreads, combine_ctas(A, BATCH * TOKENS)) combine_kernel(const __grid_constant__ CombineParams p)
{
    int64_t t;
    uint32_t u;
    my_place<A, TOKENS>(p.data, blockIdx.x, &t, &u);
    grid_dependency_wait();
    if (u >= p.data.units)
        return;
    if (A == 16 || u - threadIdx.x % 32 + 32 * accesses(A) <= p.data.units)
        combine_rows<D, A, BATCH, TOKENS, true>(p, t, u);
    else
        combine_rows<D, A, BATCH, TOKENS, false>(p, t, u);
}

struct CombineGradParams {
    const void *rows;
    const void *dy;
    const int32_t *places;
    const float *weights;
    void *drows;
    float *dweights;
    int64_t tokens, dy_stride;             // elements
    uint32_t rows_stride, drows_stride;    // elements, below 2^30
    uint32_t limit, units;
    int32_t top_k;
};

// The sums of N values each over LANES neighbouring lanes: lane l gets that of value l % N.  Half of the values change
// hands at each of the first steps, so four values take 6 exchanges over a warp, not 20.
template <int N, int LANES>
__device__ __forceinline__ float lanes_sums(float *v)
{
#pragma unroll
    for (int d = 1, n = N; n > 1; d *= 2, n /= 2) {
        const bool odd = threadIdx.x & d;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            // the even lane keeps the values whose number has this bit 0
            const float keep = odd ? v[2 * i + 1] : v[2 * i], give = odd ? v[2 * i] : v[2 * i + 1];
            v[i] = keep + __shfl_xor_sync(kFullWarp, give, d);
        }
    }
    float sum = v[0];
#pragma unroll
    for (int d = N; d < LANES; d *= 2)
        sum += __shfl_xor_sync(kFullWarp, sum, d);
    return sum;
}

// LANES threads take a token: of a warp (4, 8, 16 or 32), or the CTA (0).  A thread has HELD accesses of dy at a time, 32
// apart (LANES, where fewer); the rows of BATCH places are in flight together, and while dy is in registers each row's
// gradient is written and its product summed: one pass.  16384 x 4096 bf16, 8 places: 328 us, 103 % of the copy rate;
// 65536 x 256, 4 places: 49.7 us (91 %), 65536 x 64, 8 places: 27.3 us (80 %; the sums' exchanges), 8192 x 2049, 4 places:
// 89.7 us (50 %; instructions).
template <int D, int A, int LANES, int HELD, int BATCH>
__global__ void __launch_bounds__(kRowThreads) combine_backward_kernel(const __grid_constant__ CombineGradParams p)
{
    using T = typename Elem<D>::type;
    using B = typename Bits<A>::type;
    constexpr int V = A / static_cast<int>(sizeof(T));
    constexpr int kLanes = LANES ? LANES : 32;   // that sum by shuffles
    __shared__ float s_dot[kRowThreads / kLanes][CNS_ROUTE_MAX_TOP_K];
    const uint32_t slot = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
    const int64_t t = LANES ? static_cast<int64_t>(blockIdx.x) * (kRowThreads / kLanes) + slot : blockIdx.x;
    const bool token = t < p.tokens;
    grid_dependency_wait();
    for (int j = l; j < p.top_k; j += kLanes)
        s_dot[slot][j] = 0.f;
    __syncwarp();
    const int32_t *place = p.places + t * p.top_k;
    const float *weight = p.weights + t * p.top_k;
    const uint32_t stretch = LANES ? kLanes * HELD : blockDim.x * HELD;
    for (uint32_t u0 = 0; u0 < p.units; u0 += stretch) {   // as often in every thread
        const uint32_t u = u0 + (LANES ? 0u : slot * (32 * HELD)) + l;
        const auto mine = [&](int k) { return token && u + k * kLanes < p.units; };
        const B *from = reinterpret_cast<const B *>(static_cast<const T *>(p.dy) + t * p.dy_stride) + u;
        float dy[HELD][V];
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            B raw = B{};
            if (mine(k))
                raw = from[k * kLanes];
            unpack<D, A>(raw, dy[k]);
        }
        for (int j = 0; j < p.top_k; j += BATCH) {
            uint32_t row[BATCH];
            B raw[BATCH][HELD];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                row[i] = token && j + i < p.top_k ? static_cast<uint32_t>(place[j + i]) : 0xffffffffu;
                const T *from_row = static_cast<const T *>(p.rows) + static_cast<uint64_t>(row[i]) * p.rows_stride;
                const B *at = reinterpret_cast<const B *>(from_row) + u;
#pragma unroll
                for (int k = 0; k < HELD; ++k)
                    raw[i][k] = B{};
                if (p.dweights && row[i] < p.limit) {
#pragma unroll
                    for (int k = 0; k < HELD; ++k)
                        if (mine(k))
                            raw[i][k] = at[k * kLanes];
                }
            }
            float dot[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const bool there = row[i] < p.limit;
                if (p.drows && there) {
                    const float w = p.weights ? weight[j + i] : 1.f;
                    T *to_row = static_cast<T *>(p.drows) + static_cast<uint64_t>(row[i]) * p.drows_stride;
                    B *to = reinterpret_cast<B *>(to_row) + u;
#pragma unroll
                    for (int k = 0; k < HELD; ++k) {
                        float v[V];
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            v[e] = w * dy[k][e];
                        if (mine(k))
                            to[k * kLanes] = pack<D, A>(v);
                    }
                }
                dot[i] = 0.f;
                if (there) {
#pragma unroll
                    for (int k = 0; k < HELD; ++k) {
                        float v[V];
                        unpack<D, A>(raw[i][k], v);
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            dot[i] = fmaf(dy[k][e], v[e], dot[i]);
                    }
                }
            }
            if (p.dweights) {
                const float sum = lanes_sums<BATCH, kLanes>(dot);
                if (l < BATCH && j + static_cast<int>(l) < p.top_k)
                    s_dot[slot][j + l] += sum;
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
    for (int j = LANES ? l : threadIdx.x; j < p.top_k; j += LANES ? kLanes : blockDim.x) {
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

template <int D, int A, int BATCH, int TOKENS>
cudaError_t launch_combine_as(CombineParams &p, int sms, cudaStream_t s)
{
    tile(p.tokens, p.data.units, A, TOKENS, &p.data);   // cns_combine has seen that it fits
    uint32_t ctas = p.data.ctas;
    if constexpr (A == 16) {
        const uint32_t most = static_cast<uint32_t>(sms) * combine_ctas(A, BATCH * TOKENS);
        // whole rows of parts, so that a thread keeps its part
        ctas = std::min(ctas, std::max<uint32_t>(most / p.data.parts, 1u) * p.data.parts);
        p.step = static_cast<int64_t>(ctas / p.data.parts) * p.data.per * TOKENS;
    } else {
        p.step = p.tokens;   // one round: a warp's part is by its number
    }
    return launch<CombineParams>(combine_kernel<D, A, BATCH, TOKENS>, p, ctas, p.data.threads, s);
}

// Rows in flight a thread, by the places of a token: four of one token, or of two, with 64 registers; six with 80 where
// four would leave a second batch of one or two (16384 x 4096 bf16, 6 places: 142 us, with four 154; 3 places of two
// tokens 85.8, of one with a batch of four 89.1).  One place is best with two tokens (50.0 us; three and four spill or
// lack threads: 50.5 to 162).
template <int D>
cudaError_t launch_combine(CombineParams &p, int access, int sms, cudaStream_t s)
{
    constexpr int E = sizeof(typename Elem<D>::type);
    if (access == 16)
        return p.top_k == 1                   ? launch_combine_as<D, 16, 1, 2>(p, sms, s)
               : p.top_k == 2                 ? launch_combine_as<D, 16, 2, 2>(p, sms, s)
               : p.top_k == 3                 ? launch_combine_as<D, 16, 3, 2>(p, sms, s)
               : p.top_k == 5 || p.top_k == 6 ? launch_combine_as<D, 16, 6, 1>(p, sms, s)
                                              : launch_combine_as<D, 16, 4, 1>(p, sms, s);
    return access == 8   ? launch_combine_as<D, 8, 4, 1>(p, sms, s)
           : access == 4 ? launch_combine_as<D, 4, 4, 1>(p, sms, s)
                         : launch_combine_as<D, E, 4, 1>(p, sms, s);
}

template <int D, int A, int LANES, int HELD, int BATCH>
cudaError_t launch_grad_as(const CombineGradParams &p, cudaStream_t s)
{
    const int64_t per = kRowThreads / (LANES ? LANES : kRowThreads);
    const uint32_t threads = LANES ? kRowThreads : std::min<uint32_t>(kRowThreads, (p.units + 32 * HELD - 1) / (32 * HELD) * 32);
    return launch<CombineGradParams>(combine_backward_kernel<D, A, LANES, HELD, BATCH>, p,
                                     static_cast<uint32_t>((p.tokens + per - 1) / per), threads, s);
}

// A token's lanes: enough for the row's accesses, two each, so that few idle, few exchanges are left and few sums meet in
// shared memory.  One access a lane, or four rows at once: 65536 x 256, 4 places, 58.4 and 53.0 us against 49.7; the CTA's
// four rows at once 371 us against 328 at 16384 x 4096.
template <int D>
cudaError_t launch_combine_backward(const CombineGradParams &p, int access, cudaStream_t s)
{
    constexpr int E = sizeof(typename Elem<D>::type);
    if (access == 16)
        return p.units <= 8    ? launch_grad_as<D, 16, 4, 2, 2>(p, s)
               : p.units <= 16 ? launch_grad_as<D, 16, 8, 2, 2>(p, s)
               : p.units <= 32 ? launch_grad_as<D, 16, 16, 2, 2>(p, s)
               : p.units <= 64 ? launch_grad_as<D, 16, 32, 2, 2>(p, s)
                               : launch_grad_as<D, 16, 0, 2, 2>(p, s);
    const auto narrow = [&](auto bytes) {
        constexpr int A = bytes();
        return p.units <= 32 * accesses(A) ? launch_grad_as<D, A, 32, accesses(A), 2>(p, s)
                                           : launch_grad_as<D, A, 0, accesses(A), 2>(p, s);
    };
    return access == 8   ? narrow(std::integral_constant<int, 8>())
           : access == 4 ? narrow(std::integral_constant<int, 4>())
                         : narrow(std::integral_constant<int, E>());
}

bool sizes_ok(int64_t tokens, int64_t rows, int32_t top_k, int32_t reserved)
{
    return tokens >= 0 && rows >= 0 && top_k >= 1 && top_k <= CNS_ROUTE_MAX_TOP_K && tokens <= 0x7fffffff / top_k &&
           reserved == 0;
}

// A matrix's stride (`packed` where it is 0); false if it is too small, or too large for kernels that multiply it in
// 32 bits.
template <class S>
bool stride_ok(int64_t given, int64_t packed, S *stride)
{
    const int64_t s = given ? given : packed;
    *stride = static_cast<S>(s);
    return s >= packed && s <= CNS_ROWS_MAX_STRIDE;
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
    if (!tile(p.tokens, d->row_bytes / access, access, 1, &p.data))
        return CNS_ERR_INVALID_VALUE;
    if (scales) {
        const int a = access_bytes(address(p.scales) | address(p.row_scales) | d->scale_bytes | p.scales_stride | p.row_scales_stride);
        p.scale_access = a == 16 ? 16 : a >= 4 ? 4 : 1;
        if (!tile(p.tokens, d->scale_bytes / p.scale_access, p.scale_access, 1, &p.scale))
            return CNS_ERR_INVALID_VALUE;
    }
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
                    p, p.data.ctas + p.scale.ctas, threads, to_stream(d->stream)));
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
    if (!tile(p.tokens, c->width * e / access, access, 1, &p.data))
        return CNS_ERR_INVALID_VALUE;
    DeviceInfo dev;
    if (int rc = current_device(&dev))
        return rc;
    if (p.tokens == 0)
        return CNS_SUCCESS;
    cudaStream_t s = to_stream(c->stream);
    CNS_CUDA(c->dtype == CNS_DT_F32    ? launch_combine<CNS_DT_F32>(p, access, dev.sm_count, s)
             : c->dtype == CNS_DT_BF16 ? launch_combine<CNS_DT_BF16>(p, access, dev.sm_count, s)
                                       : launch_combine<CNS_DT_F16>(p, access, dev.sm_count, s));
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
