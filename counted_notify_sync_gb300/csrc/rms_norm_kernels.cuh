// rms_norm_kernels.cuh -- the kernels of the root-mean-square norm
// (cns_rms_norm, cns_rms_norm_backward); rms_norm_{f32,bf16,f16}.cu instantiate
// them, a type each.
//
//   h = round(x + residual),  r = 1 / sqrt(mean h^2 + eps),  y = h r gain,
//   per block of columns: s from the largest |y|, q = e4m3(y / s)
//   dx = dh + r g - h r^3 mean(g h) with g = gain dy;  dgain = sum over rows dy h r
//
// G threads take a row and hold it: one pass over the operands.  A thread has HOLD vectors of 16 bytes, G vectors
// apart; a block of 32 columns or more is then the vectors of neighbouring lanes of one warp.  WIDE rows are read
// and written by vectors, others by elements, at the same places.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "rows_device.cuh"

namespace cns {

struct NormParams {
    const void *x;
    const void *residual;
    const void *gain;
    void *h;
    void *y;
    uint8_t *q;
    void *scales;
    int64_t rows, x_stride, residual_stride, h_stride, y_stride, q_stride, scales_stride;
    int32_t width, gain_dtype, block, power;
    float eps;
};

struct NormGradParams {
    const void *h;
    const void *gain;
    const void *dy;
    const void *dh;
    void *dx;
    float *parts;   // [CTAs][width]: the CTAs' sums of dgain
    int64_t rows, h_stride, dy_stride, dh_stride, dx_stride;
    int32_t width, gain_dtype;
    float eps;
};

// Most CTAs of a gradient, each of which leaves a part of dgain: four to an SM.
constexpr int kNormMaxParts = 4 * kStepMaxCtas;

template <int D> __host__ __device__ constexpr int norm_vec() { return 16 / static_cast<int>(sizeof(typename Elem<D>::type)); }

// The vector of columns e .. of a row; what lies past the row is 0.
template <int D, bool WIDE>
__device__ __forceinline__ uint4 load_vec(const void *row, int e, int width)
{
    using T = typename Elem<D>::type;
    const T *a = static_cast<const T *>(row) + e;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (WIDE) {
        if (e < width)
            raw = *reinterpret_cast<const uint4 *>(a);
    } else {
        T *to = reinterpret_cast<T *>(&raw);
#pragma unroll
        for (int i = 0; i < norm_vec<D>(); ++i)
            if (e + i < width)
                to[i] = a[i];
    }
    return raw;
}

template <int D, bool WIDE>
__device__ __forceinline__ void store_vec(void *row, int e, int width, const uint4 &raw)
{
    using T = typename Elem<D>::type;
    T *a = static_cast<T *>(row) + e;
    if constexpr (WIDE) {
        if (e < width)
            *reinterpret_cast<uint4 *>(a) = raw;
    } else {
        const T *from = reinterpret_cast<const T *>(&raw);
#pragma unroll
        for (int i = 0; i < norm_vec<D>(); ++i)
            if (e + i < width)
                a[i] = from[i];
    }
}

// N columns of the gain from column e on, in 32 bits.
template <int N, bool WIDE>
__device__ __forceinline__ void load_gain(const void *gain, int dtype, int e, int width, float *v)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = gain ? 0.f : 1.f;
    if (!gain || e >= width)
        return;
    if constexpr (WIDE) {
        if (dtype == CNS_DT_F32) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                unpack<CNS_DT_F32, 16>(*reinterpret_cast<const uint4 *>(static_cast<const float *>(gain) + e + i), v + i);
        } else {
            const auto raw = *reinterpret_cast<const typename Bits<2 * N>::type *>(static_cast<const uint16_t *>(gain) + e);
            if (dtype == CNS_DT_BF16)
                unpack<CNS_DT_BF16, 2 * N>(raw, v);
            else
                unpack<CNS_DT_F16, 2 * N>(raw, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (e + i < width)
                v[i] = dtype == CNS_DT_F32    ? static_cast<const float *>(gain)[e + i]
                       : dtype == CNS_DT_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(gain)[e + i])
                                              : __half2float(static_cast<const __half *>(gain)[e + i]);
    }
}

// The sum of `a` and the largest `b` (as whole numbers: magnitudes, NaN above all) over the G threads of a row.  The
// halves of `s` alternate from call to call, so one barrier each is enough.
template <int G>
__device__ __forceinline__ void join_row(float &a, uint32_t &b, uint2 (*s)[32], int turn)
{
#pragma unroll
    for (int d = (G < 32 ? G : 32) / 2; d > 0; d >>= 1) {
        a += __shfl_xor_sync(kFullWarp, a, d);
        b = max(b, __shfl_xor_sync(kFullWarp, b, d));
    }
    if constexpr (G > 32) {
        if (threadIdx.x % 32 == 0)
            s[turn & 1][threadIdx.x / 32] = make_uint2(__float_as_uint(a), b);
        __syncthreads();
        a = 0.f;
        b = 0u;
#pragma unroll
        for (int i = 0; i < G / 32; ++i) {
            const uint2 v = s[turn & 1][i];
            a += __uint_as_float(v.x);
            b = max(b, v.y);
        }
    }
}

// Two e4m3 values, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float low, float high)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(high), "f"(low));
    return r;
}

// Threads of a CTA whose rows take G threads each.
__host__ __device__ constexpr int norm_threads(int g) { return g < 128 ? 128 : g; }

template <int D, bool WIDE, int G, int HOLD>
__global__ void __launch_bounds__(norm_threads(G)) rms_norm_kernel(const __grid_constant__ NormParams p)
{
    using T = typename Elem<D>::type;
    constexpr int V = norm_vec<D>();
    constexpr int kGroups = norm_threads(G) / G;
    __shared__ uint2 s_join[2][32];
    const int g = threadIdx.x % G, group = threadIdx.x / G;
    grid_dependency_wait();
    // the gain: in registers, or, where a CTA of 512 threads or more has none left, loaded for each row
    constexpr bool kHeld = G < 512;
    float held_gain[kHeld ? HOLD : 1][V];
    if constexpr (kHeld) {
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            load_gain<V, WIDE>(p.gain, p.gain_dtype, (j * G + g) * V, p.width, held_gain[j]);
    }
    const auto gain_of = [&](int j, float *v) {
        if constexpr (kHeld) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = held_gain[j][i];
        } else {
            load_gain<V, WIDE>(p.gain, p.gain_dtype, (j * G + g) * V, p.width, v);
        }
    };
    int turn = 0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kGroups; first < p.rows;
         first += static_cast<int64_t>(gridDim.x) * kGroups, ++turn) {
        const int64_t row = first + group;
        const int width = row < p.rows ? p.width : 0;   // past the last row, a row without columns
        uint4 held[HOLD];
        const T *x = static_cast<const T *>(p.x) + row * p.x_stride;
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            held[j] = load_vec<D, WIDE>(x, (j * G + g) * V, width);
        if (p.residual) {
            const T *residual = static_cast<const T *>(p.residual) + row * p.residual_stride;
            uint4 more[HOLD];
#pragma unroll
            for (int j = 0; j < HOLD; ++j)
                more[j] = load_vec<D, WIDE>(residual, (j * G + g) * V, width);
            T *h = static_cast<T *>(p.h) + row * p.h_stride;
#pragma unroll
            for (int j = 0; j < HOLD; ++j) {
                float a[V], b[V];
                unpack<D, 16>(held[j], a);
                unpack<D, 16>(more[j], b);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    a[i] += b[i];
                held[j] = pack<D, 16>(a);
                store_vec<D, WIDE>(h, (j * G + g) * V, width, held[j]);
            }
        }
        const bool whole = p.q && p.block == 0;
        float sum = 0.f;
        uint32_t top = 0u;
#pragma unroll
        for (int j = 0; j < HOLD; ++j) {
            float v[V];
            unpack<D, 16>(held[j], v);
#pragma unroll
            for (int i = 0; i < V; ++i)
                sum = fmaf(v[i], v[i], sum);
            if (whole) {
                float gain[V];
                gain_of(j, gain);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    top = max(top, __float_as_uint(fabsf(v[i] * gain[i])));
            }
        }
        join_row<G>(sum, top, s_join, turn);
        const float r = 1.f / sqrtf(sum / static_cast<float>(p.width) + p.eps);
        if (whole)
            top = __float_as_uint(fabsf(__uint_as_float(top) * r));
        T *y = static_cast<T *>(p.y) + row * p.y_stride;
#pragma unroll
        for (int j = 0; j < HOLD; ++j) {
            const int e = (j * G + g) * V;
            float v[V], gain[V];
            unpack<D, 16>(held[j], v);
            gain_of(j, gain);
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = v[i] * r * gain[i];
            if (p.y)
                store_vec<D, WIDE>(y, e, width, pack<D, 16>(v));
            if (!p.q)
                continue;
            uint32_t m = top;
            if (p.block) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    m = max(m, __float_as_uint(fabsf(v[i])));
                for (int d = p.block / V / 2; d > 0; d >>= 1)
                    m = max(m, __shfl_xor_sync(kFullWarp, m, d));
            }
            const bool finite = m < 0x7f800000u;
            float inverse;
            const bool writes = p.block ? e < width && e % p.block == 0 : e == 0 && width > 0;
            const int64_t at = row * p.scales_stride + (p.block ? e / p.block : 0);
            if (p.power) {
                // m = c 2^a with c in [1, 2), 448 = 1.75 * 2^8: the exponent is a - 8, and one more where c > 1.75
                const int biased = max(static_cast<int>(m >> 23) - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
                inverse = __uint_as_float(finite ? static_cast<uint32_t>(254 - biased) << 23 : 0x7fffffffu);
                if (writes)
                    static_cast<uint8_t *>(p.scales)[at] = finite ? static_cast<uint8_t>(biased) : 255u;
            } else {
                const float scale = finite ? fmaxf(__uint_as_float(m) / 448.f, 1.17549435e-38f) : __uint_as_float(0x7fffffffu);
                inverse = 1.f / scale;
                if (writes)
                    static_cast<float *>(p.scales)[at] = scale;
            }
            uint32_t bytes[V / 4];
#pragma unroll
            for (int i = 0; i < V; i += 4)
                bytes[i / 4] = e4m3_pair(v[i] * inverse, v[i + 1] * inverse) |
                               e4m3_pair(v[i + 2] * inverse, v[i + 3] * inverse) << 16;
            uint8_t *q = p.q + row * p.q_stride + e;
            if constexpr (WIDE) {
                if (e < width) {
                    if constexpr (V == 8)
                        *reinterpret_cast<uint2 *>(q) = make_uint2(bytes[0], bytes[1]);
                    else
                        *reinterpret_cast<uint32_t *>(q) = bytes[0];
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e + i < width)
                        q[i] = static_cast<uint8_t>(bytes[i / 4] >> (8 * (i % 4)));
            }
        }
    }
}

template <int D, bool WIDE, int G, int HOLD>
__global__ void __launch_bounds__(norm_threads(G)) rms_norm_backward_kernel(const __grid_constant__ NormGradParams p)
{
    using T = typename Elem<D>::type;
    constexpr int V = norm_vec<D>();
    constexpr int kGroups = norm_threads(G) / G;
    __shared__ float2 s_join[2][32];
    // where a CTA takes several rows at once, their sums of dgain at the end, [groups][width]; from 512 threads on,
    // whose registers do not hold them, the sums all along, [HOLD][V][threads]
    extern __shared__ float s_gain[];
    constexpr bool kHeld = G < 512;
    const int g = threadIdx.x % G, group = threadIdx.x / G;
    grid_dependency_wait();
    float held_gain[kHeld ? HOLD : 1][V], dgain[kHeld ? HOLD : 1][V];
#pragma unroll
    for (int j = 0; j < HOLD; ++j) {
        if constexpr (kHeld)
            load_gain<V, WIDE>(p.gain, p.gain_dtype, (j * G + g) * V, p.width, held_gain[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (kHeld)
                dgain[j][i] = 0.f;
            else
                s_gain[(j * V + i) * G + g] = 0.f;
        }
    }
    const auto gain_of = [&](int j, float *v) {
        if constexpr (kHeld) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = held_gain[j][i];
        } else {
            load_gain<V, WIDE>(p.gain, p.gain_dtype, (j * G + g) * V, p.width, v);
        }
    };
    const float share = 1.f / static_cast<float>(p.width);
    int turn = 0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kGroups; first < p.rows;
         first += static_cast<int64_t>(gridDim.x) * kGroups, ++turn) {
        const int64_t row = first + group;
        const int width = row < p.rows ? p.width : 0;
        const T *h = static_cast<const T *>(p.h) + row * p.h_stride, *dy = static_cast<const T *>(p.dy) + row * p.dy_stride;
        uint4 held[HOLD], grad[HOLD];
#pragma unroll
        for (int j = 0; j < HOLD; ++j) {
            held[j] = load_vec<D, WIDE>(h, (j * G + g) * V, width);
            grad[j] = load_vec<D, WIDE>(dy, (j * G + g) * V, width);
        }
        float sum = 0.f, inner = 0.f;
#pragma unroll
        for (int j = 0; j < HOLD; ++j) {
            float a[V], b[V], gain[V];
            unpack<D, 16>(held[j], a);
            unpack<D, 16>(grad[j], b);
            gain_of(j, gain);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sum = fmaf(a[i], a[i], sum);
                inner = fmaf(b[i] * gain[i], a[i], inner);
            }
        }
#pragma unroll
        for (int d = (G < 32 ? G : 32) / 2; d > 0; d >>= 1) {
            sum += __shfl_xor_sync(kFullWarp, sum, d);
            inner += __shfl_xor_sync(kFullWarp, inner, d);
        }
        if constexpr (G > 32) {
            if (threadIdx.x % 32 == 0)
                s_join[turn & 1][threadIdx.x / 32] = make_float2(sum, inner);
            __syncthreads();
            sum = inner = 0.f;
#pragma unroll
            for (int i = 0; i < G / 32; ++i) {
                sum += s_join[turn & 1][i].x;
                inner += s_join[turn & 1][i].y;
            }
        }
        const float r = 1.f / sqrtf(sum * share + p.eps);
        const float back = inner * share * r * r;   // of h r
        const T *dh = static_cast<const T *>(p.dh) + row * p.dh_stride;
        T *dx = static_cast<T *>(p.dx) + row * p.dx_stride;
#pragma unroll
        for (int j = 0; j < HOLD; ++j) {
            float a[V], b[V], v[V], gain[V];
            unpack<D, 16>(held[j], a);
            unpack<D, 16>(grad[j], b);
            gain_of(j, gain);
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = 0.f;
            if (p.dh)
                unpack<D, 16>(load_vec<D, WIDE>(dh, (j * G + g) * V, width), v);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float &sum_of = kHeld ? dgain[kHeld ? j : 0][i] : s_gain[(j * V + i) * G + g];
                if (width)
                    sum_of = fmaf(b[i], a[i] * r, sum_of);
                v[i] = fmaf(r, fmaf(-a[i], back, b[i] * gain[i]), v[i]);
            }
            store_vec<D, WIDE>(dx, (j * G + g) * V, width, pack<D, 16>(v));
        }
    }
    if (!p.parts)
        return;
    float *part = p.parts + static_cast<int64_t>(blockIdx.x) * p.width;
    if constexpr (kGroups > 1) {
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = (j * G + g) * V + i;
                if (e < p.width)
                    s_gain[group * p.width + e] = dgain[kHeld ? j : 0][i];
            }
        __syncthreads();
        for (int e = threadIdx.x; e < p.width; e += norm_threads(G)) {
            float v = 0.f;
            for (int i = 0; i < kGroups; ++i)
                v += s_gain[i * p.width + e];
            part[e] = v;
        }
    } else {
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = (j * G + g) * V + i;
                if (e < p.width)
                    part[e] = kHeld ? dgain[kHeld ? j : 0][i] : s_gain[(j * V + i) * G + g];
            }
    }
}

template <class P>
cudaError_t launch_norm(void (*kernel)(P), const P &p, int g, int ctas, size_t smem, cudaStream_t s)
{
    cudaLaunchAttribute early;
    cudaLaunchConfig_t cfg = early_launch(&early);
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(norm_threads(g));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// CTAs of a call: as many as rows need, up to `most`.
inline int norm_ctas(int64_t rows, int g, int most)
{
    const int64_t groups = norm_threads(g) / g, ctas = (rows + groups - 1) / groups;
    return static_cast<int>(ctas < most ? ctas : most);
}

// The threads of a row and the vectors each holds, by the row's vectors.  With 8-bit blocks a row has a warp at least
// (a block's vectors are neighbouring lanes').
template <int D, bool WIDE>
cudaError_t launch_forward(const NormParams &p, int sms, cudaStream_t s)
{
    const int vecs = (p.width + norm_vec<D>() - 1) / norm_vec<D>();
    const auto go = [&](auto kernel, int g) {
        return launch_norm<NormParams>(kernel, p, g, norm_ctas(p.rows, g, sms * 16), 0, s);
    };
    if (vecs <= 16 && !(p.q && p.block))
        return go(rms_norm_kernel<D, WIDE, 8, 2>, 8);
    if (vecs <= 64)
        return go(rms_norm_kernel<D, WIDE, 32, 2>, 32);
    if (vecs <= 128)
        return go(rms_norm_kernel<D, WIDE, 32, 4>, 32);
    if (vecs <= 256)
        return go(rms_norm_kernel<D, WIDE, 128, 2>, 128);
    if (vecs <= 512)
        return go(rms_norm_kernel<D, WIDE, 128, 4>, 128);
    if (vecs <= 1024)
        return go(rms_norm_kernel<D, WIDE, 256, 4>, 256);
    if (vecs <= 2048)
        return go(rms_norm_kernel<D, WIDE, 512, 4>, 512);
    if (vecs <= 4096)
        return go(rms_norm_kernel<D, WIDE, 1024, 4>, 1024);
    return go(rms_norm_kernel<D, WIDE, 1024, norm_vec<D>() == 8 ? 4 : 8>, 1024);   // 32768 columns in 32 bits
}

template <int D, bool WIDE, int G, int HOLD>
cudaError_t launch_backward_as(const NormGradParams &p, int most, int *parts, cudaStream_t s)
{
    constexpr int kGroups = norm_threads(G) / G;
    const auto kernel = rms_norm_backward_kernel<D, WIDE, G, HOLD>;
    size_t smem = kGroups > 1 ? sizeof(float) * kGroups * p.width : 0;
    if constexpr (G >= 512) {
        smem = sizeof(float) * HOLD * norm_vec<D>() * G;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess)
            return e;
    }
    *parts = norm_ctas(p.rows, G, most < kNormMaxParts ? most : kNormMaxParts);
    return launch_norm<NormGradParams>(kernel, p, G, *parts, smem, s);
}

template <int D, bool WIDE>
cudaError_t launch_backward(const NormGradParams &p, int sms, int *parts, cudaStream_t s)
{
    constexpr int V = norm_vec<D>();
    const int vecs = (p.width + V - 1) / V;
    if (vecs <= 16)
        return launch_backward_as<D, WIDE, 8, 2>(p, 4 * sms, parts, s);
    if (vecs <= 64)
        return launch_backward_as<D, WIDE, 32, 2>(p, 4 * sms, parts, s);
    if (vecs <= 128)
        return launch_backward_as<D, WIDE, 32, 4>(p, 4 * sms, parts, s);
    if (vecs <= 256)
        return launch_backward_as<D, WIDE, 128, 2>(p, 4 * sms, parts, s);
    if (vecs <= 512)
        return launch_backward_as<D, WIDE, 128, 4>(p, 4 * sms, parts, s);
    if (vecs <= 1024)
        return launch_backward_as<D, WIDE, 256, 4>(p, 2 * sms, parts, s);
    if (vecs <= 2048)
        return launch_backward_as<D, WIDE, 512, 4>(p, 2 * sms, parts, s);
    if (vecs <= 4096 || V == 8)
        return launch_backward_as<D, WIDE, 1024, 4>(p, sms, parts, s);
    return launch_backward_as<D, WIDE, 1024, V == 8 ? 4 : 8>(p, sms, parts, s);
}

// A type's kernels (rms_norm_*.cu); `parts`: how many parts of dgain the call leaves.
cudaError_t launch_rms_norm_f32(const NormParams &p, bool wide, int sms, cudaStream_t s);
cudaError_t launch_rms_norm_bf16(const NormParams &p, bool wide, int sms, cudaStream_t s);
cudaError_t launch_rms_norm_f16(const NormParams &p, bool wide, int sms, cudaStream_t s);
cudaError_t launch_rms_norm_backward_f32(const NormGradParams &p, bool wide, int sms, int *parts, cudaStream_t s);
cudaError_t launch_rms_norm_backward_bf16(const NormGradParams &p, bool wide, int sms, int *parts, cudaStream_t s);
cudaError_t launch_rms_norm_backward_f16(const NormGradParams &p, bool wide, int sms, int *parts, cudaStream_t s);

}  // namespace cns
