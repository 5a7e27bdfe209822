// rms_norm_kernels.cuh -- the kernels of the root-mean-square norm
// (cns_rms_norm, cns_rms_norm_backward); rms_norm_{f32,bf16,f16}.cu instantiate
// them, a type each.
//
//   h = round(x + residual),  r = 1 / sqrt(mean h^2 + eps),  y = h r gain,
//   per block of columns: s from the largest |y|, q = e4m3(y / s)
//   dx = dh + r g - h r^3 mean(g h) with g = gain dy;  dgain = sum over rows dy h r
//
// A group of threads takes a row, one pass over the operands: a thread has HOLD vectors of 16 bytes, as far apart as the
// group is large, so that a block of 32 columns or more is the vectors of neighbouring lanes of one warp.  As many CTAs
// as the GPU holds go through the rows in steps, so a CTA's sums of dgain stay on the SM, and the next rows are on their
// way while one is worked on: WIDE rows, whose vectors are aligned, are copied to shared memory ahead (every thread
// copies what it will read itself, so no thread waits for another's copies), others pass through shared memory element
// by element, in neighbouring lanes' order on the global side and by vectors on the registers'.
//
// Bound by HBM where a residual or y comes along, by instructions (14.6 an element of bf16, 63 % of the issue slots, by 16
// warps an SM) where rows only become e4m3 with scales in 32 bits.  16384 x 4096 bf16: with a residual to h and y 84.0 us
// (94 % of the copy rate), and e4m3 with powers of two by 32 columns too 99.4 us (90 %), from x to y 41.7 us (95 %), to
// e4m3 alone 41.0 us (73 %), with powers of two 32.4 us (92 %); the gradient 82.3 us (96 %), in 32 bits at 2048 columns
// 78.1 us (101 %).  8192 x 2049 (narrow): 49.8 us with e4m3 (45 %), gradient 61.0 us (32 %).  More than 8192 columns of 16
// bits: 4096 x 16384 90.8 us to h and y (87 %), gradient 146 (54 %), 2048 x 32768 86.5 and 297 (27 %; registers spill).
// The products and sums by pairs (f32x2 instructions), the gain in registers and threads that fit the row took the norm
// with all its outputs from 36 instructions an element to 23, the gradient from 36 to 19.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

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
    float *dgain;   // NULL: not wanted
    float *parts;   // [CTAs][width]: the CTAs' sums of dgain; of one CTA dgain itself
    int64_t rows, h_stride, dy_stride, dh_stride, dx_stride;
    int32_t width, gain_dtype;
    bool joined;    // whether a grid that joins the parts follows
    float eps;
};

// Most CTAs of a gradient, each of which leaves a part of dgain: 512 threads to an SM in CTAs of 160 or more.
constexpr int kNormMaxParts = 3 * kStepMaxCtas;
// Rows that a group of a gradient has at least, so that few parts are left to join: as many as it takes for no more CTAs
// than SMs, four at most; four where one CTA then has all rows and no join follows.  In us, with one / two / four at least:
//   f32    64 x 1000  3.38 / 3.71 / 4.57    256 x 1000  3.66 / 4.01 / 4.76    777 x 1000  5.31 / 5.05 / 4.97
//         256 x 4096  6.15 / 6.02 / 7.31
//   bf16   64 x 1000  4.05 / 4.58 / 5.60    777 x 1000  5.42 / 4.90 / 5.88   2000 x 1000  6.65 / 6.54 / 6.10
//           8 x 4096  5.16 / 5.67 / 6.64    256 x 4096  8.50 / 6.72 / 7.35
// and with eight less for 777 x 4096 bf16 alone (9.8, 10.7 to 11.0 with fewer).  The rule's three rows take 777 x 1000 f32
// in 4.53.
__host__ __device__ constexpr int norm_least_rows(int64_t rows, int groups, int sms)
{
    const int64_t ctas = (rows + groups - 1) / groups, each = (ctas + sms - 1) / sms;
    return ctas <= 4 || each > 4 ? 4 : static_cast<int>(each);
}

// Dynamic shared memory that every kernel here may be launched with.
constexpr int kNormMaxSmem = 200 * 1024;

template <int D> __host__ __device__ constexpr int norm_vec() { return 16 / static_cast<int>(sizeof(typename Elem<D>::type)); }

// A thread's vectors of a row at any address.  The lanes of a warp that share a row read or write neighbouring elements and
// exchange them through `scratch`, 16 bytes a thread.
template <int D, int G, int HOLD>
__device__ __forceinline__ void load_narrow(const void *row, int width, uint4 *scratch, uint4 *to)
{
    using T = typename Elem<D>::type;
    constexpr int V = norm_vec<D>(), L = G < 32 ? G : 32;
    const int g = threadIdx.x % G, l = g % L;
    const T *from = static_cast<const T *>(row) + (g - l) * V + l;
    T *s = reinterpret_cast<T *>(scratch + (threadIdx.x - l));
    T v[HOLD][V];
#pragma unroll
    for (int j = 0; j < HOLD; ++j) {
        const int first = (j * G + g - l) * V;   // of the lanes' stretch
        if (first + L * V <= width) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[j][i] = from[j * G * V + i * L];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[j][i] = first + i * L + l < width ? from[j * G * V + i * L] : T(0.f);
        }
    }
#pragma unroll
    for (int j = 0; j < HOLD; ++j) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < V; ++i)
            s[i * L + l] = v[j][i];
        __syncwarp();
        to[j] = scratch[threadIdx.x];
    }
}

// One vector of N-byte elements from every thread: its column is e, the threads of a row's warp hold neighbouring ones.
template <class T, int V, int L, class Raw>
__device__ __forceinline__ void store_narrow(T *row, int e, int width, uint4 *scratch, const Raw &raw)
{
    static_assert(sizeof(Raw) == V * sizeof(T), "one vector");
    const int lane = threadIdx.x & 31, l = lane % L;
    Raw *mine = reinterpret_cast<Raw *>(scratch + (threadIdx.x - lane)) + lane;   // within the warp's 512 bytes
    const T *s = reinterpret_cast<const T *>(mine - l);
    __syncwarp();
    *mine = raw;
    __syncwarp();
    const int first = e - l * V;   // of the lanes' stretch
    row += first + l;
    if (first + L * V <= width) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            row[i * L] = s[i * L + l];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (first + i * L + l < width)
                row[i * L] = s[i * L + l];
    }
}

template <int D, bool WIDE, int L>
__device__ __forceinline__ void store_vec(void *row, int e, int width, uint4 *scratch, const uint4 &raw)
{
    using T = typename Elem<D>::type;
    if constexpr (WIDE) {
        if (e < width)
            *reinterpret_cast<uint4 *>(static_cast<T *>(row) + e) = raw;
    } else {
        store_narrow<T, norm_vec<D>(), L>(static_cast<T *>(row), e, width, scratch, raw);
    }
}

// A copy of 16 bytes to shared memory that the thread does not wait for; zeros where there is nothing to copy (then no
// byte of `from` is read).
__device__ __forceinline__ void copy_ahead(uint4 *to, const void *from, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                 "l"(from), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LATER>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LATER) : "memory"); }

// A vector as pairs, for the instructions that work on two numbers at once.
template <int D>
__device__ __forceinline__ void unpack_pairs(const uint4 &raw, float2 *v)
{
    float f[norm_vec<D>()];
    unpack<D, 16>(raw, f);
#pragma unroll
    for (int i = 0; i < norm_vec<D>() / 2; ++i)
        v[i] = make_float2(f[2 * i], f[2 * i + 1]);
}

template <int D>
__device__ __forceinline__ uint4 pack_pairs(const float2 *v)
{
    float f[norm_vec<D>()];
#pragma unroll
    for (int i = 0; i < norm_vec<D>() / 2; ++i) {
        f[2 * i] = v[i].x;
        f[2 * i + 1] = v[i].y;
    }
    return pack<D, 16>(f);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Rows of G threads: a CTA has GROUPS groups of them, each for a row at a time.
template <int G, int GROUPS>
struct Group {
    static constexpr int kThreads = G * GROUPS, kLanes = G < 32 ? G : 32;   // kLanes: of a warp
    static __device__ __forceinline__ int rank() { return threadIdx.x % G; }
    static __device__ __forceinline__ int number() { return threadIdx.x / G; }
    static __device__ __forceinline__ void sync()
    {
        if constexpr (GROUPS == 1) {
            __syncthreads();
        } else {
            static_assert(GROUPS <= 4, "a barrier each");
            const int n = number();   // barriers by number: the CTA then has five, not all sixteen
            if (n == 0)
                asm volatile("bar.sync 1, %0;" ::"n"(G) : "memory");
            else if (n == 1)
                asm volatile("bar.sync 2, %0;" ::"n"(G) : "memory");
            else if (n == 2)
                asm volatile("bar.sync 3, %0;" ::"n"(G) : "memory");
            else
                asm volatile("bar.sync 4, %0;" ::"n"(G) : "memory");
        }
    }
};

// One operand's rows as a thread goes through them: its first vector of the row at hand (the row's first column where
// rows are narrow).  With DEPTH > 0 its vectors come through shared memory, the DEPTH rows from that one on being on
// their way or there.
template <int D, bool WIDE, int G, int HOLD, int DEPTH, int THREADS>
struct Operand {
    using T = typename Elem<D>::type;
    static constexpr int V = norm_vec<D>();
    const T *at;      // the next row to copy, or to load
    int64_t apart;    // elements to the thread's next row
    uint4 *ring;      // [DEPTH][HOLD][THREADS], the thread's own

    __device__ __forceinline__ void start(const void *base, int64_t row, int64_t stride, int64_t step, uint4 *s)
    {
        at = static_cast<const T *>(base) + row * stride + (WIDE ? static_cast<int>(threadIdx.x) % G * V : 0);
        apart = step * stride;
        ring = s + threadIdx.x;
    }
    // into stage `stage`; `width`: 0 for a row past the last, whose vectors are zeros
    __device__ __forceinline__ void copy(int stage, int width)
    {
        const int left = width - static_cast<int>(threadIdx.x) % G * V;
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            copy_ahead(ring + (stage * HOLD + j) * THREADS, at + j * G * V, j * G * V < left);
        at += apart;
    }
    // `scratch`: as load_narrow
    __device__ __forceinline__ void get(int stage, int width, uint4 *scratch, uint4 *to)
    {
        if constexpr (DEPTH > 0) {
#pragma unroll
            for (int j = 0; j < HOLD; ++j)
                to[j] = ring[(stage * HOLD + j) * THREADS];
        } else if constexpr (WIDE) {
            const int left = width - static_cast<int>(threadIdx.x) % G * V;
#pragma unroll
            for (int j = 0; j < HOLD; ++j) {
                to[j] = make_uint4(0u, 0u, 0u, 0u);
                if (j * G * V < left)
                    to[j] = *reinterpret_cast<const uint4 *>(at + j * G * V);
            }
            at += apart;
        } else {
            load_narrow<D, G, HOLD>(at, width, scratch, to);
            at += apart;
        }
    }
};

// One result's rows: the row's first column.
template <class T>
struct Result {
    T *at;
    int64_t apart;
    __device__ __forceinline__ void start(void *base, int64_t row, int64_t stride, int64_t step)
    {
        at = static_cast<T *>(base) + row * stride;
        apart = step * stride;
    }
    __device__ __forceinline__ void next() { at += apart; }
};

// N columns of the gain from column e on, in 32 bits.
template <int N, bool WIDE>
__device__ __forceinline__ void load_gain(const void *gain, int dtype, int e, int width, float2 *pairs)
{
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = gain ? 0.f : 1.f;
    if (gain && e < width) {
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
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
        pairs[i] = make_float2(v[2 * i], v[2 * i + 1]);
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Values of a row's warps to be joined: of each group from a multiple of four on.  The places between a group's last warp
// and the next group's first are left as they are, and no result depends on them: a group has no barrier with the
// others, so nothing that another group's threads would have to write first is read.
template <int G, int GROUPS>
struct Joined {
    static constexpr int kWarps = G / 32, kRoom = kWarps > 4 ? (kWarps + 3) / 4 * 4 : 4, kSize = G > 32 ? kRoom * GROUPS : 4;
    float4 s[2][kSize / 4];   // the halves alternate from row to row, so one barrier each is enough
    __device__ __forceinline__ void put(int turn, float v)
    {
        if (threadIdx.x % 32 == 0)
            reinterpret_cast<float *>(s[turn & 1])[Group<G, GROUPS>::number() * kRoom + threadIdx.x % G / 32] = v;
    }
    // the values of a group's kWarps warps, joined
#pragma nv_exec_check_disable
    template <class F>
    static __host__ __device__ __forceinline__ float fold(const float4 *of, F join)
    {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kRoom / 4; ++i) {
            const float4 w = of[i];
            float part = 4 * i + 1 < kWarps ? join(w.x, w.y) : w.x;
            if (4 * i + 2 < kWarps)
                part = join(part, 4 * i + 3 < kWarps ? join(w.z, w.w) : w.z);
            v = i ? join(v, part) : part;
        }
        return v;
    }
    template <class F>
    __device__ __forceinline__ float get(int turn, F join) const
    {
        return fold(s[turn & 1] + Group<G, GROUPS>::number() * (kRoom / 4), join);
    }
};

template <int G, class F>
__device__ __forceinline__ float join_lanes(float v, F join)
{
#pragma unroll
    for (int d = (G < 32 ? G : 32) / 2; d > 0; d >>= 1)
        v = join(v, __shfl_xor_sync(kFullWarp, v, d));
    return v;
}

struct Add {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Largest {
    __device__ __forceinline__ float operator()(float a, float b) const { return max_nan(a, b); }
};

// A value joined over a row's threads.
template <int G, int GROUPS, class F>
__device__ __forceinline__ float join_row(float v, F join, Joined<G, GROUPS> &s, int turn)
{
    v = join_lanes<G>(v, join);
    if constexpr (G > 32) {
        s.put(turn, v);
        Group<G, GROUPS>::sync();
        v = s.get(turn, join);
    }
    return v;
}

// Two sums over a row's threads, with one barrier.
template <int G, int GROUPS>
__device__ __forceinline__ void sum_row(float &a, float &b, Joined<G, GROUPS> &sa, Joined<G, GROUPS> &sb, int turn)
{
    a = join_lanes<G>(a, Add());
    b = join_lanes<G>(b, Add());
    if constexpr (G > 32) {
        sa.put(turn, a);
        sb.put(turn, b);
        Group<G, GROUPS>::sync();
        a = sa.get(turn, Add());
        b = sb.get(turn, Add());
    }
}

// Two e4m3 values, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float low, float high)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(high), "f"(low));
    return r;
}

// 1 / sqrt(m) to within a unit in the last place: an approximation and a step of Newton's.
__device__ __forceinline__ float root_reciprocal(float m)
{
    const float r = rsqrtf(m);
    return m < INFINITY ? fmaf(0.5f * r, fmaf(-m * r, r, 1.f), r) : r;
}

// m / 448 for a magnitude whose quotient is a normal number, rounded to the nearest: the product with the reciprocal, off by
// less than 1.25 units in the last place, and its remainder times that reciprocal.  The remainder is less than nine of its
// least steps, so exact, and the quotient is a fourteenth of a unit or more away from where the rounding changes.
__device__ __forceinline__ float over_448(float m)
{
    const float c = 1.f / 448.f, q = m * c;
    return fmaf(fmaf(-448.f, q, m), c, q);
}

// v / s for V numbers no larger than 448 s (or so), s >= 2^-126 or NaN, each rounded to 32 bits, so that a quotient halfway
// between two e4m3 values is found there.  In two forms: `any_quotients` for every s, and `quotients` for those that
// `usual` says, half the instructions, with the same e4m3 values.
//
// Markstein's correction, twice: the product with the rounded reciprocal is off by less than 1.5 units in the last place, the
// first correction leaves one of the two neighbours of the quotient, whose remainder is then exact, and the second rounds
// it to the nearest.  The quotients are negated up to there, not the reciprocal, so that a remainder of 0 keeps a zero's
// sign.  Remainders below the subnormal numbers would be lost, so a small s is scaled up, and v with it; where a quotient
// is too small for that to help, it is less than half of the least e4m3.
template <int V>
__device__ __forceinline__ void any_quotients(float2 *v, float s)
{
    const float up = s < 0x1p-60f ? 0x1p64f : 1.f;
    s *= up;
    const float2 back = both(-__frcp_rn(s)), ss = both(s);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const float2 of = __fmul2_rn(v[i], both(up));
        float2 q = __fmul2_rn(of, back);
        q = __ffma2_rn(__ffma2_rn(ss, q, of), back, q);
        v[i] = __fmul2_rn(__ffma2_rn(__ffma2_rn(ss, q, of), back, q), both(-1.f));
    }
}

// The reciprocal in two numbers, hi below it and lo the rest (both positive, which keeps a zero's sign), and v hi + (v lo):
// the quotient to within 2^-42 of itself, then rounded.  That gives another e4m3 value than the rounded quotient only where
// the quotient is as near to the rounding border next to a tie: with v = V 2^i, s = S 2^k (V, S of 24 bits) and ties of
// four bits after the point, K / 16, where S (K 2^20 +- 1) is within 2^49 2^-42 of a multiple of 2^24, so S within 128 of
// one of 2^20.  Such S, one in 4096, are not `usual`, nor those whose lo, or remainder, would be below the normal numbers.
// 16384 x 4096 bf16 to e4m3 alone, a scale for 128 columns, when this came: 42.7 us, by any_quotients alone 51.8, by one
// product with the reciprocal (whose ties fall either way) 38.8.
__device__ __forceinline__ bool usual(float s)
{
    const uint32_t bits = __float_as_uint(s);
    return bits - 0x21800000u < 0x3c000000u /* 2^-60 .. 2^60 */ && ((bits + 128u) & 0xfffffu) > 256u;
}

template <int V>
__device__ __forceinline__ void quotients(float2 *v, float s)
{
    float x;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(s));   // off by up to two units in the last place: below 1 / s by
    const float hi = __uint_as_float(__float_as_uint(x) - 3u);   // one to five of them, e 2^-20.6 at most
    const float e = fmaf(-s, hi, 1.f), lo = fmaf(e, e, e) * hi;
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
        v[i] = __ffma2_rn(v[i], both(hi), __fmul2_rn(v[i], both(lo)));
}

// V numbers as e4m3, four in a word.
template <int V>
__device__ __forceinline__ void to_e4m3(const float2 *v, uint32_t *bytes)
{
#pragma unroll
    for (int i = 0; i < V / 2; i += 2)
        bytes[i / 2] = e4m3_pair(v[i].x, v[i].y) | e4m3_pair(v[i + 1].x, v[i + 1].y) << 16;
}

// Groups of a CTA: enough for 128 threads where a warp or less takes a row, for 256 in the gradient, whose CTAs each
// leave a part to join.
__host__ __device__ constexpr int norm_groups(int g, bool grad)
{
    return grad ? (g < 256 ? 256 / g : 1) : g <= 32 ? 128 / g : 1;
}

// CTAs to an SM that its registers and shared memory are shared out for: 768 threads with two vectors each, 512 of the
// gradient or with more vectors.
__host__ __device__ constexpr int norm_ctas_per_sm(int g, int hold, bool grad)
{
    const int threads = g * norm_groups(g, grad), all = grad || hold > 2 ? 512 : 768;
    return threads > all ? 1 : all / threads;
}

// Whether the gradient's sums of dgain stay in registers; else they are in shared memory.
__host__ __device__ constexpr bool norm_sums_in_registers(int g, int hold) { return g * hold <= 2048 && hold <= 4; }

// Rows on their way ahead of the one at hand, of `operands` tensors each (3: the gradient): two, one of a norm with a
// residual; none where the shared memory lacks the room.  More of them cost time, presumably because the DRAM's pages are
// left and opened again in between: 16384 x 4096 bf16 takes the norm with a residual 84.0 us with one, 85.2 with two and
// 89.2 with four (and with e4m3 99.4, 103.5 and 106.5), without one 47.2, 41.7 and (three) 44.9; its gradient 89.5, 82.6
// and (four) 88.5.
__host__ __device__ constexpr int norm_depth(bool wide, int g, int hold, int operands)
{
    const bool grad = operands == 3;
    const int depth = operands == 2 ? 1 : 2, threads = g * norm_groups(g, grad) * norm_ctas_per_sm(g, hold, grad);
    return !wide || (grad && !norm_sums_in_registers(g, hold)) || 16 * threads * hold * depth * operands > 192 * 1024 ? 0 : depth;
}

// RESIDUAL: whether there is one (narrow rows: whether there may be one).
template <int D, bool WIDE, int G, int HOLD, bool RESIDUAL>
__global__ void __launch_bounds__(G * norm_groups(G, false), norm_ctas_per_sm(G, HOLD, false))
rms_norm_kernel(const __grid_constant__ NormParams p)
{
    using T = typename Elem<D>::type;
    constexpr int V = norm_vec<D>(), kGroups = norm_groups(G, false), kDepth = norm_depth(WIDE, G, HOLD, RESIDUAL ? 2 : 1);
    using Row = Group<G, kGroups>;
    constexpr int kThreads = Row::kThreads, kLanes = Row::kLanes;
    constexpr bool kGain = G * HOLD <= 1024;   // the gain stays in registers
    const bool add = RESIDUAL && (WIDE || p.residual);
    extern __shared__ uint4 s_rows[];   // the operands' rings; narrow rows: 16 bytes a thread
    __shared__ Joined<G, kGroups> s_first, s_second;
    const int g = Row::rank();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kGroups + Row::number();
    Operand<D, WIDE, G, HOLD, kDepth, kThreads> x, residual;
    x.start(p.x, row, p.x_stride, step, s_rows);
    residual.start(p.residual, row, p.residual_stride, step, s_rows + kDepth * HOLD * kThreads);
    const auto copy = [&](int stage, int64_t of) {
        const int width = of < p.rows ? p.width : 0;   // past the last row, a row without columns
        x.copy(stage, width);
        if constexpr (RESIDUAL)
            residual.copy(stage, width);
        copies_end();
    };
    grid_dependency_wait();
    if constexpr (kDepth > 0) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
            copy(d, row + d * step);
    }
    Result<T> h, y;
    Result<uint8_t> q;
    h.start(p.h, row, p.h_stride, step);
    y.start(p.y, row, p.y_stride, step);
    q.start(p.q, row, p.q_stride, step);
    float2 gain[HOLD][V / 2];
    if constexpr (kGain) {
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            load_gain<V, WIDE>(p.gain, p.gain_dtype, (j * G + g) * V, p.width, gain[j]);
    }
    const float share = 1.f / static_cast<float>(p.width);
    const bool whole = p.block == 0;
    // The lanes of a block, which of them writes its scale, and that scale's number.  (The vectors of a thread are a
    // multiple of 128 columns apart where there are blocks, so this holds for each of them.)
    const int lanes = p.block / V, shift = p.block ? 31 - __clz(p.block) : 0;
    const bool writes = p.block ? (g * V & (p.block - 1)) == 0 : g == 0;
    int64_t scale_at = row * p.scales_stride + (g * V >> shift);
    int stage = 0, turn = 0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kGroups; first < p.rows; first += step, row += step, ++turn) {
        const int width = row < p.rows ? p.width : 0;
        if constexpr (kDepth > 0)
            copies_wait<(kDepth > 0 ? kDepth - 1 : 0)>();
        uint4 held[HOLD];
        x.get(stage, width, s_rows, held);
        if (add) {
            uint4 more[HOLD];
            residual.get(stage, width, s_rows, more);
#pragma unroll
            for (int j = 0; j < HOLD; ++j) {
                float2 a[V / 2], b[V / 2];
                unpack_pairs<D>(held[j], a);
                unpack_pairs<D>(more[j], b);
#pragma unroll
                for (int i = 0; i < V / 2; ++i)
                    a[i] = __fadd2_rn(a[i], b[i]);
                held[j] = pack_pairs<D>(a);
                store_vec<D, WIDE, kLanes>(h.at, (j * G + g) * V, width, s_rows, held[j]);
            }
            h.next();
        }
        if constexpr (kDepth > 0) {
            copy(stage, row + kDepth * step);   // into the stage just read
            stage = stage + 1 == kDepth ? 0 : stage + 1;
        }
        float2 v[HOLD][V / 2], sums = both(0.f);
#pragma unroll
        for (int j = 0; j < HOLD; ++j) {
            unpack_pairs<D>(held[j], v[j]);
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                sums = __ffma2_rn(v[j][i], v[j][i], sums);
        }
        const float sum = join_row<G, kGroups>(sums.x + sums.y, Add(), s_first, turn);
        const float r = root_reciprocal(fmaf(sum, share, p.eps));
#pragma unroll
        for (int j = 0; j < HOLD; ++j) {
            if constexpr (!kGain)
                load_gain<V, WIDE>(p.gain, p.gain_dtype, (j * G + g) * V, p.width, gain[j]);
#pragma unroll
            for (int i = 0; i < V / 2; ++i)   // h r is no more than the root of the width; h times the gain may overflow
                v[j][i] = __fmul2_rn(__fmul2_rn(v[j][i], both(r)), gain[j][i]);
            if (p.y)
                store_vec<D, WIDE, kLanes>(y.at, (j * G + g) * V, width, s_rows, pack_pairs<D>(v[j]));
        }
        if (p.q) {
            float largest[HOLD];
#pragma unroll
            for (int j = 0; j < HOLD; ++j) {
                largest[j] = 0.f;
#pragma unroll
                for (int i = 0; i < V / 2; ++i)
                    largest[j] = max_nan(largest[j], max_nan(fabsf(v[j][i].x), fabsf(v[j][i].y)));
            }
            if (whole) {
                float top = largest[0];
#pragma unroll
                for (int j = 1; j < HOLD; ++j)
                    top = max_nan(top, largest[j]);
                top = join_row<G, kGroups>(top, Largest(), s_second, turn);
#pragma unroll
                for (int j = 0; j < HOLD; ++j)
                    largest[j] = top;
            } else {
                for (int d = 1; d < lanes; d *= 2)
#pragma unroll
                    for (int j = 0; j < HOLD; ++j)
                        largest[j] = max_nan(largest[j], __shfl_xor_sync(kFullWarp, largest[j], d));
            }
            const auto write = [&](int j) { return writes && (j * G + g) * V < width && (j == 0 || !whole); };
            const auto at = [&](int j) { return scale_at + (j * G * V >> shift); };
            if (p.power) {
#pragma unroll
                for (int j = 0; j < HOLD; ++j) {
                    // m = c 2^a with c in [1, 2), 448 = 1.75 * 2^8: the exponent is a - 8, and one more where c > 1.75
                    const float m = largest[j];
                    const int biased = max(static_cast<int>((__float_as_uint(m) + 0x1fffffu) >> 23) - 8, 0);
                    const bool finite = m < INFINITY;
                    if (write(j))
                        static_cast<uint8_t *>(p.scales)[at(j)] = finite ? static_cast<uint8_t>(biased) : 255u;
                    const float inverse = __uint_as_float(finite ? static_cast<uint32_t>(254 - biased) << 23 : 0x7fffffffu);
#pragma unroll
                    for (int i = 0; i < V / 2; ++i)
                        v[j][i] = __fmul2_rn(v[j][i], both(inverse));   // exact
                }
            } else {
                bool fast = true;
#pragma unroll
                for (int j = 0; j < HOLD; ++j) {
                    constexpr float kLeast = 1.17549435e-38f;   // 2^-126
                    const float m = largest[j];
                    largest[j] = m <= 448.f * kLeast ? kLeast : m < INFINITY ? over_448(m) : __uint_as_float(0x7fffffffu);
                    if (write(j))
                        static_cast<float *>(p.scales)[at(j)] = largest[j];
                    fast = fast && (usual(largest[j]) || m == 0.f);   // zeros: columns past the last among them
                }
                if (fast) {
#pragma unroll
                    for (int j = 0; j < HOLD; ++j)
                        quotients<V>(v[j], largest[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < HOLD; ++j)
                        any_quotients<V>(v[j], largest[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < HOLD; ++j) {
                const int e = (j * G + g) * V;
                uint32_t bytes[V / 4];
                to_e4m3<V>(v[j], bytes);
                typename Bits<V>::type raw;
                if constexpr (V == 8)
                    raw = make_uint2(bytes[0], bytes[1]);
                else
                    raw = bytes[0];
                if constexpr (!WIDE)
                    store_narrow<uint8_t, V, kLanes>(q.at, e, width, s_rows, raw);
                else if (e < width)
                    *reinterpret_cast<typename Bits<V>::type *>(q.at + e) = raw;
            }
        }
        y.next();
        q.next();
        scale_at += step * p.scales_stride;
    }
    if constexpr (kDepth > 0)
        copies_wait<0>();
}

template <int D, bool WIDE, int G, int HOLD>
__global__ void __launch_bounds__(G * norm_groups(G, true), norm_ctas_per_sm(G, HOLD, true))
rms_norm_backward_kernel(const __grid_constant__ NormGradParams p)
{
    using T = typename Elem<D>::type;
    constexpr int V = norm_vec<D>(), kGroups = norm_groups(G, true), kDepth = norm_depth(WIDE, G, HOLD, 3);
    using Row = Group<G, kGroups>;
    constexpr int kThreads = Row::kThreads, kLanes = Row::kLanes;
    constexpr bool kGain = HOLD <= 2, kRegisters = norm_sums_in_registers(G, HOLD);   // the gain and the sums of dgain
    static_assert(kRegisters || kGroups == 1, "several rows and sums in shared memory");
    // The operands' rings; narrow rows: 16 bytes a thread.  Then the sums of dgain where the registers do not have them,
    // [HOLD][V][G].  At the end, where a CTA takes several rows at once, [groups][width] of these sums from the start on.
    extern __shared__ uint4 s_rows[];
    float *s_gain = reinterpret_cast<float *>(s_rows + (WIDE ? 0 : kThreads));
    __shared__ Joined<G, kGroups> s_first, s_second;
    const int g = Row::rank();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kGroups + Row::number();
    Operand<D, WIDE, G, HOLD, kDepth, kThreads> h, dy, dh;
    h.start(p.h, row, p.h_stride, step, s_rows);
    dy.start(p.dy, row, p.dy_stride, step, s_rows + kDepth * HOLD * kThreads);
    dh.start(p.dh, row, p.dh_stride, step, s_rows + 2 * kDepth * HOLD * kThreads);
    const auto copy = [&](int stage, int64_t of) {
        const int width = of < p.rows ? p.width : 0;
        h.copy(stage, width);
        dy.copy(stage, width);
        if (p.dh)
            dh.copy(stage, width);
        copies_end();
    };
    grid_dependency_wait();
    if constexpr (kDepth > 0) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
            copy(d, row + d * step);
    }
    if (p.joined)
        grid_launch_dependents();   // the join of the parts, which sets up meanwhile
    Result<T> dx;
    dx.start(p.dx, row, p.dx_stride, step);
    float2 gain[HOLD][V / 2], dgain[kRegisters ? HOLD : 1][V / 2];
#pragma unroll
    for (int j = 0; j < HOLD; ++j) {
        if constexpr (kGain)
            load_gain<V, WIDE>(p.gain, p.gain_dtype, (j * G + g) * V, p.width, gain[j]);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (kRegisters)
                dgain[j][i] = both(0.f);
            else
                s_gain[(j * V + 2 * i) * G + g] = s_gain[(j * V + 2 * i + 1) * G + g] = 0.f;
        }
    }
    const float share = 1.f / static_cast<float>(p.width);
    int stage = 0, turn = 0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kGroups; first < p.rows; first += step, row += step, ++turn) {
        const int width = row < p.rows ? p.width : 0;
        if constexpr (kDepth > 0)
            copies_wait<(kDepth > 0 ? kDepth - 1 : 0)>();
        uint4 held[HOLD], grad[HOLD], more[HOLD];
        h.get(stage, width, s_rows, held);
        dy.get(stage, width, s_rows, grad);
        if (p.dh)
            dh.get(stage, width, s_rows, more);
        if constexpr (kDepth > 0) {
            copy(stage, row + kDepth * step);   // into the stage just read
            stage = stage + 1 == kDepth ? 0 : stage + 1;
        }
        float2 sums = both(0.f), inners = both(0.f);
#pragma unroll
        for (int j = 0; j < HOLD; ++j) {
            float2 a[V / 2], b[V / 2];
            unpack_pairs<D>(held[j], a);
            unpack_pairs<D>(grad[j], b);
            if constexpr (!kGain)
                load_gain<V, WIDE>(p.gain, p.gain_dtype, (j * G + g) * V, p.width, gain[j]);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                sums = __ffma2_rn(a[i], a[i], sums);
                inners = __ffma2_rn(__fmul2_rn(b[i], gain[j][i]), a[i], inners);
            }
        }
        float sum = sums.x + sums.y, inner = inners.x + inners.y;
        sum_row<G, kGroups>(sum, inner, s_first, s_second, turn);
        const float r = root_reciprocal(fmaf(sum, share, p.eps));
        const float2 back = both(-(inner * share) * r * r), rs = both(r), mine = both(width ? r : 0.f);
#pragma unroll
        for (int j = 0; j < HOLD; ++j) {
            float2 a[V / 2], b[V / 2], v[V / 2];
            unpack_pairs<D>(held[j], a);
            unpack_pairs<D>(grad[j], b);
            if constexpr (!kGain)
                load_gain<V, WIDE>(p.gain, p.gain_dtype, (j * G + g) * V, p.width, gain[j]);
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                v[i] = both(0.f);
            if (p.dh)
                unpack_pairs<D>(more[j], v);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 unit = __fmul2_rn(a[i], mine);   // past the last row 0
                if constexpr (kRegisters) {
                    dgain[j][i] = __ffma2_rn(b[i], unit, dgain[j][i]);
                } else {
                    float *sum_of = s_gain + (j * V + 2 * i) * G + g;
                    sum_of[0] = fmaf(b[i].x, unit.x, sum_of[0]);
                    sum_of[G] = fmaf(b[i].y, unit.y, sum_of[G]);
                }
                v[i] = __ffma2_rn(rs, __ffma2_rn(a[i], back, __fmul2_rn(b[i], gain[j][i])), v[i]);
            }
            store_vec<D, WIDE, kLanes>(dx.at, (j * G + g) * V, width, s_rows, pack_pairs<D>(v));
        }
        dx.next();
    }
    if constexpr (kDepth > 0)
        copies_wait<0>();
    if (!p.parts)
        return;
    float *part = p.parts + static_cast<int64_t>(blockIdx.x) * p.width;
    const auto sum_of = [&](int j, int i) {
        if constexpr (kRegisters)
            return i % 2 ? dgain[j][i / 2].y : dgain[j][i / 2].x;
        else
            return s_gain[(j * V + i) * G + g];
    };
    if constexpr (kGroups > 1) {
        __syncthreads();
        float *sums = reinterpret_cast<float *>(s_rows);
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = (j * G + g) * V + i;
                if (e < p.width)
                    sums[Row::number() * p.width + e] = sum_of(j, i);
            }
        __syncthreads();
        for (int e = threadIdx.x; e < p.width; e += kThreads) {
            float v = 0.f;
            for (int i = 0; i < kGroups; ++i)
                v += sums[i * p.width + e];
            part[e] = v;
        }
    } else {
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = (j * G + g) * V + i;
                if (e < p.width)
                    part[e] = sum_of(j, i);
            }
    }
}

// CTAs of a call whose CTAs take `groups` rows at once: as many as the rows need (`each` of them at least to a group),
// `most` at most.
inline int norm_ctas(int64_t rows, int groups, int each, int most)
{
    const int64_t per = static_cast<int64_t>(groups) * each, need = (rows + per - 1) / per;
    return static_cast<int>(need < most ? need : most);
}

template <class P>
cudaError_t launch_norm(void (*kernel)(P), const P &p, int threads, int ctas, int smem, cudaStream_t s)
{
    if (smem > 47 * 1024) {   // the kernels have up to 512 bytes of their own
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxSmem);
        if (e != cudaSuccess)
            return e;
    }
    cudaLaunchAttribute early;
    cudaLaunchConfig_t cfg = early_launch(&early);
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, bool WIDE, int G, int HOLD, bool RESIDUAL>
cudaError_t launch_forward_as(const NormParams &p, int sms, cudaStream_t s)
{
    constexpr int kGroups = norm_groups(G, false), kThreads = G * kGroups, kOperands = RESIDUAL ? 2 : 1;
    constexpr int kSmem = 16 * kThreads * (WIDE ? norm_depth(WIDE, G, HOLD, kOperands) * kOperands * HOLD : 1);
    return launch_norm<NormParams>(rms_norm_kernel<D, WIDE, G, HOLD, RESIDUAL>, p, kThreads,
                                   norm_ctas(p.rows, kGroups, 1, sms * norm_ctas_per_sm(G, HOLD, false)), kSmem, s);
}

template <int D, bool WIDE, int G, int HOLD>
cudaError_t launch_backward_as(const NormGradParams &p, int sms, int *parts, cudaStream_t s)
{
    constexpr int kGroups = norm_groups(G, true), kThreads = G * kGroups;
    int smem = 16 * kThreads * (WIDE ? norm_depth(WIDE, G, HOLD, 3) * (p.dh ? 3 : 2) * HOLD : 1);
    if (!norm_sums_in_registers(G, HOLD))
        smem += 4 * HOLD * norm_vec<D>() * kThreads;
    if (kGroups > 1)
        smem = std::max(smem, 4 * kGroups * p.width);
    const int most = std::min<int>(sms, kStepMaxCtas) * norm_ctas_per_sm(G, HOLD, true);
    static_assert(norm_ctas_per_sm(G, HOLD, true) * kStepMaxCtas <= kNormMaxParts, "room for the parts");
    *parts = norm_ctas(p.rows, kGroups, norm_least_rows(p.rows, kGroups, sms), most);
    NormGradParams with = p;
    with.joined = p.dgain && *parts > 1;
    if (!with.joined)
        with.parts = p.dgain;
    return launch_norm<NormGradParams>(rms_norm_backward_kernel<D, WIDE, G, HOLD>, with, kThreads, *parts, smem, s);
}

// Calls what(G, HOLD) for rows of `vecs` vectors.  Two vectors a thread up to 1024 (8192 columns of 16 bits), and as few
// warps as hold them; four vectors beyond.  Blocks of columns need a warp to a row at least (a block's vectors are
// neighbouring lanes').  `few`: four vectors a thread from 128 on; where little memory traffic comes with much arithmetic
// it pays that half as many threads do what each does once a row (16384 x 4096 bf16 to e4m3 alone 41.0 us, with two
// vectors 47.4, with powers of two 32.4 and 40.6; with a residual and y, when it was tried, 101.2 against 98.9).
template <int V, bool FEW, class F>
cudaError_t with_shape(int vecs, bool blocks, bool few, F what)
{
#define CNS_NORM_SHAPE(G, HOLD) \
    if (vecs <= G * HOLD)       \
        return what(std::integral_constant<int, G>(), std::integral_constant<int, HOLD>())
    if (!blocks)
        CNS_NORM_SHAPE(8, 2);
    CNS_NORM_SHAPE(32, 2);
    CNS_NORM_SHAPE(64, 2);
    if constexpr (FEW) {
        if (few) {
            CNS_NORM_SHAPE(64, 4);
            CNS_NORM_SHAPE(96, 4);
            CNS_NORM_SHAPE(128, 4);
            CNS_NORM_SHAPE(160, 4);
            CNS_NORM_SHAPE(192, 4);
            CNS_NORM_SHAPE(224, 4);
            CNS_NORM_SHAPE(256, 4);
        }
    }
    CNS_NORM_SHAPE(96, 2);
    CNS_NORM_SHAPE(128, 2);
    CNS_NORM_SHAPE(160, 2);
    CNS_NORM_SHAPE(192, 2);
    CNS_NORM_SHAPE(224, 2);
    CNS_NORM_SHAPE(256, 2);
    CNS_NORM_SHAPE(320, 2);
    CNS_NORM_SHAPE(384, 2);
    CNS_NORM_SHAPE(448, 2);
    CNS_NORM_SHAPE(512, 2);
    CNS_NORM_SHAPE(512, 4);
    CNS_NORM_SHAPE(1024, 4);
    if constexpr (V == 4)
        CNS_NORM_SHAPE(1024, 8);   // 32768 columns in 32 bits
    return cudaErrorInvalidValue;
#undef CNS_NORM_SHAPE
}

template <int D, bool WIDE, bool RESIDUAL>
cudaError_t launch_forward_with(const NormParams &p, int sms, cudaStream_t s)
{
    constexpr int V = norm_vec<D>();
    return with_shape<V, WIDE && !RESIDUAL>((p.width + V - 1) / V, p.q && p.block, p.q && !p.y, [&](auto g, auto hold) {
        return launch_forward_as<D, WIDE, g(), hold(), RESIDUAL>(p, sms, s);
    });
}

template <int D, bool WIDE>
cudaError_t launch_forward(const NormParams &p, int sms, cudaStream_t s)
{
    if constexpr (WIDE)
        if (!p.residual)
            return launch_forward_with<D, WIDE, false>(p, sms, s);
    return launch_forward_with<D, WIDE, true>(p, sms, s);
}

template <int D, bool WIDE>
cudaError_t launch_backward(const NormGradParams &p, int sms, int *parts, cudaStream_t s)
{
    constexpr int V = norm_vec<D>();
    return with_shape<V, false>((p.width + V - 1) / V, false, false, [&](auto g, auto hold) {
        return launch_backward_as<D, WIDE, g(), hold()>(p, sms, parts, s);
    });
}

// A type's kernels (rms_norm_*.cu); `parts`: how many parts of dgain the call leaves.
cudaError_t launch_rms_norm_f32(const NormParams &p, bool wide, int sms, cudaStream_t s);
cudaError_t launch_rms_norm_bf16(const NormParams &p, bool wide, int sms, cudaStream_t s);
cudaError_t launch_rms_norm_f16(const NormParams &p, bool wide, int sms, cudaStream_t s);
cudaError_t launch_rms_norm_backward_f32(const NormGradParams &p, bool wide, int sms, int *parts, cudaStream_t s);
cudaError_t launch_rms_norm_backward_bf16(const NormGradParams &p, bool wide, int sms, int *parts, cudaStream_t s);
cudaError_t launch_rms_norm_backward_f16(const NormGradParams &p, bool wide, int sms, int *parts, cudaStream_t s);

}  // namespace cns
