// gradclip.cu -- the global gradient norm over many tensors, and clipping by
// it (cns_grad_norm, cns_grad_clip).
//
//   norm = sqrt(sum over all tensors of x^2)   (or the largest |x|)
//   out  = x * min(1, max_norm / (norm + eps))
//
// Tensors are cut into tiles of kTileBytes at 16-byte boundaries of the
// address space (so a tile's vectors are aligned wherever its tensor starts;
// only a tensor's first and last vector can be partial).  One warp takes one
// tile.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "cns.h"
#include "cns_host.h"
#include "step_device.cuh"

namespace cns {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
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

struct GradParams {
    const GradEntry *table;   // in the workspace, when it is not among the arguments
    uint32_t *header;
    float *norm;
    uint64_t timeout_ns;
    int32_t count;
    uint32_t tiles;
    float max_norm, eps;
};

// The kernel's arguments: the table of up to N tensors among them (N = 0: in
// the workspace).
template <int N> struct GradArgs {
    GradParams p;
    GradEntry e[N];
};
template <> struct GradArgs<0> {
    GradParams p;
};

template <int N>
__device__ __forceinline__ GradEntry entry_of(const GradArgs<N> &a, int i)
{
    if constexpr (N > 0)
        return a.e[i];
    else
        return a.p.table[i];
}

template <int N>
__device__ __forceinline__ uint32_t tile0_of(const GradArgs<N> &a, int i)
{
    if constexpr (N > 0)
        return a.e[i].tile0;
    else
        return a.p.table[i].tile0;
}

// A table of more tensors than fit the arguments goes to the workspace as the
// arguments of launches of this kernel: no staging buffer, and nothing that a
// graph capture would lose.
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

// Largest i with tile0 <= tile (tensors without elements have
// no tiles and are not in the table).
template <int N>
__device__ __forceinline__ int find_tensor(const GradArgs<N> &a, uint32_t tile)
{
    int lo = 0, hi = a.p.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tile0_of(a, mid) <= tile)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ uint4 ld_stream(uint64_t a)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(a)
                 : "memory");
    return v;
}

// The elements of one 16-byte vector as floats.
template <int D> struct Vec {
    using T = typename Elem<D>::type;
    static constexpr int N = 16 / static_cast<int>(sizeof(T));
    static __device__ __forceinline__ void unpack(const uint4 &v, float *f)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (D == CNS_DT_F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (D == CNS_DT_BF16) {
                    f[2 * i] = __uint_as_float(w[i] << 16);
                    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                } else {
                    const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                    f[2 * i] = g.x;
                    f[2 * i + 1] = g.y;
                }
            }
        }
    }
};

// The calling lane's vectors of a tile.  Vectors that the tensor covers only in
// part are loaded element by element; what the tensor does not cover is 0.
template <int D>
__device__ __forceinline__ uint4 load_part(uint64_t a, uint64_t src, uint64_t end)
{
    using T = typename Elem<D>::type;
    union { uint4 v; uint16_t h[8]; uint32_t w[4]; } u;
    u.v = make_uint4(0u, 0u, 0u, 0u);
    if (a + 16 <= src || a >= end)
        return u.v;
#pragma unroll
    for (int i = 0; i < Vec<D>::N; ++i) {
        const uint64_t at = a + i * sizeof(T);
        if (at >= src && at < end) {
            if constexpr (sizeof(T) == 4)
                u.w[i] = *reinterpret_cast<const uint32_t *>(at);
            else
                u.h[i] = *reinterpret_cast<const uint16_t *>(at);
        }
    }
    return u.v;
}

template <int D>
__device__ __forceinline__ void load_tile(uint64_t base, uint64_t src, uint64_t end, uint4 *v)
{
    const uint64_t mine = base + (threadIdx.x & 31u) * 16u;
    if (base >= src && base + kTileBytes <= end) {
#pragma unroll
        for (int j = 0; j < kLaneVecs; ++j)
            v[j] = ld_stream(mine + j * 512);
    } else {
#pragma unroll
        for (int j = 0; j < kLaneVecs; ++j) {
            const uint64_t a = mine + j * 512;
            v[j] = a >= src && a + 16 <= end ? ld_stream(a) : load_part<D>(a, src, end);
        }
    }
}

// A tile's part of the norm for the calling lane: the sum of its squares, or
// its largest magnitude (as integers, so that NaN is above inf).
template <int NORM, int D>
__device__ __forceinline__ float tile_part(const uint4 *v)
{
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kLaneVecs; ++j) {
        float f[Vec<D>::N];
        Vec<D>::unpack(v[j], f);
#pragma unroll
        for (int i = 0; i < Vec<D>::N; ++i) {
            if constexpr (NORM == CNS_NORM_L2)
                acc[i & 3] = fmaf(f[i], f[i], acc[i & 3]);
            else
                acc[i & 3] = __uint_as_float(max(__float_as_uint(acc[i & 3]), __float_as_uint(fabsf(f[i]))));
        }
    }
    if constexpr (NORM == CNS_NORM_L2)
        return (acc[0] + acc[1]) + (acc[2] + acc[3]);
    else
        return __uint_as_float(max(max(__float_as_uint(acc[0]), __float_as_uint(acc[1])),
                                   max(__float_as_uint(acc[2]), __float_as_uint(acc[3]))));
}

// The running part over tiles, warps and CTAs: in 64 bits.
template <int NORM>
__device__ __forceinline__ double join(double a, double b)
{
    if constexpr (NORM == CNS_NORM_L2)
        return a + b;
    else   // non-negative: ordered as integers, NaN above inf
        return __longlong_as_double(max(__double_as_longlong(a), __double_as_longlong(b)));
}

template <int NORM>
__device__ __forceinline__ double warp_join(double v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v = join<NORM>(v, __shfl_xor_sync(kFullWarp, v, d));
    return v;
}

template <int D>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (D == CNS_DT_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Store n = N (4 or 8) values to dst in type D, as wide as its alignment lets;
// `from` and `to` bound the values that the tensor has.
template <int D, int N>
__device__ __forceinline__ void store_vec(uint64_t dst, const float *f, int from, int to)
{
    using T = typename Elem<D>::type;
    if (from == 0 && to == N && dst % 16 == 0) {
        if constexpr (D == CNS_DT_F32) {
            if constexpr (N == 8) {
                if (dst % 32 == 0) {   // one 32-byte sector
                    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(f[0]),
                                 "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                                 : "memory");
                    return;
                }
            }
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<float4 *>(dst + 4 * i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
            return;
        } else if constexpr (N == 8) {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(pack2<D>(f[0], f[1]), pack2<D>(f[2], f[3]),
                                                         pack2<D>(f[4], f[5]), pack2<D>(f[6], f[7]));
            return;
        }
    }
    if constexpr (D != CNS_DT_F32 && N == 4) {
        if (from == 0 && to == N && dst % 8 == 0) {
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<D>(f[0], f[1]), pack2<D>(f[2], f[3]));
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i >= from && i < to)
            reinterpret_cast<T *>(dst)[i] = Elem<D>::put(f[i]);
}

template <int DS, int DD>
__device__ __forceinline__ void scale_tile(const GradEntry &t, uint64_t base, uint64_t end, const uint4 *v, float factor)
{
    using S = typename Elem<DS>::type;
    using T = typename Elem<DD>::type;
    constexpr int N = Vec<DS>::N;
    const uint64_t mine = base + (threadIdx.x & 31u) * 16u;
#pragma unroll
    for (int j = 0; j < kLaneVecs; ++j) {
        const uint64_t a = mine + j * 512;
        if (a + 16 <= t.src || a >= end)
            continue;
        float f[N];
        Vec<DS>::unpack(v[j], f);
#pragma unroll
        for (int i = 0; i < N; ++i)
            f[i] *= factor;
        const int from = a < t.src ? static_cast<int>((t.src - a) / sizeof(S)) : 0;
        const int to = a + 16 > end ? static_cast<int>((end - a) / sizeof(S)) : N;
        // the vector's first element may lie before the tensor: its place is then never written
        const int64_t first = (static_cast<int64_t>(a) - static_cast<int64_t>(t.src)) / static_cast<int64_t>(sizeof(S));
        store_vec<DD, N>(t.dst + first * static_cast<int64_t>(sizeof(T)), f, from, to);
    }
}

template <int D>
__device__ __forceinline__ void rescale_tile(const GradEntry &t, uint64_t base, uint64_t end, float factor)
{
    uint4 v[kLaneVecs];
    load_tile<D>(base, t.src, end, v);
    switch (t.types >> 8) {
    case CNS_DT_F32: scale_tile<D, CNS_DT_F32>(t, base, end, v, factor); break;
    case CNS_DT_BF16: scale_tile<D, CNS_DT_BF16>(t, base, end, v, factor); break;
    default: scale_tile<D, CNS_DT_F16>(t, base, end, v, factor); break;
    }
}

template <int NORM, bool CLIP, int N>
__global__ void __launch_bounds__(kThreads, 1) grad_kernel(const __grid_constant__ GradArgs<N> a)
{
    const GradParams &p = a.p;
    __shared__ double s_part[kWarps];
    __shared__ float s_factor;
    __shared__ int s_stop;
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t first = warp * gridDim.x + blockIdx.x, step = kWarps * gridDim.x;
    uint64_t tag = 0;
    bool stop = false;
    if (warp == 0) {
        tag = static_cast<uint64_t>(ld_relaxed_gpu(p.header + kStepEpochWord)) + 1u;
        stop = ld_relaxed_gpu(p.header + kStepStatusWord + 1) != 0u;   // an earlier call failed
    }

    double part = 0.0;
    int at = 0;
    uint32_t next = 0;   // first tile after tensor `at`
    GradEntry t;
    uint64_t base = 0, end = 0;
    // move to `tile`'s tensor
    auto seek = [&](uint32_t tile) {
        at = find_tensor(a, tile);
        t = entry_of(a, at);
        next = at + 1 < p.count ? tile0_of(a, at + 1) : p.tiles;
        end = t.src + static_cast<uint64_t>(t.elems) * ((t.types & 0xffu) == CNS_DT_F32 ? 4 : 2);
    };
    uint32_t tile = first;
    for (; tile < p.tiles; tile += step) {
        if (tile >= next)
            seek(tile);
        base = (t.src & ~15ull) + static_cast<uint64_t>(tile - t.tile0) * kTileBytes;
        uint4 v[kLaneVecs];
        float f;
        switch (t.types & 0xffu) {
        case CNS_DT_F32:
            load_tile<CNS_DT_F32>(base, t.src, end, v);
            f = tile_part<NORM, CNS_DT_F32>(v);
            break;
        case CNS_DT_BF16:
            load_tile<CNS_DT_BF16>(base, t.src, end, v);
            f = tile_part<NORM, CNS_DT_BF16>(v);
            break;
        default:
            load_tile<CNS_DT_F16>(base, t.src, end, v);
            f = tile_part<NORM, CNS_DT_F16>(v);
            break;
        }
        part = join<NORM>(part, static_cast<double>(f));
    }
    part = warp_join<NORM>(part);
    if (lane == 0)
        s_part[warp] = part;
    __syncthreads();
    if (warp == 0) {
        part = warp_join<NORM>(s_part[lane]);
        if (gridDim.x > 1 && !stop) {
            if (lane == 0)
                st_slot(p.header, blockIdx.x, static_cast<uint64_t>(__double_as_longlong(part)), tag);
            part = 0.0;
            // CTA c's part goes to lane c % 32 in the order of c: the same sum every time
            stop = wait_slots(p.header, gridDim.x, tag, p.timeout_ns, [&](uint32_t, uint64_t v) {
                part = join<NORM>(part, __longlong_as_double(static_cast<long long>(v)));
            });
            part = warp_join<NORM>(part);
            if (!stop && blockIdx.x == 0 && lane == 0)
                st_relaxed_gpu(p.header + kStepEpochWord, static_cast<uint32_t>(tag));
        }
        if (lane == 0) {
            const float norm = static_cast<float>(NORM == CNS_NORM_L2 ? sqrt(part) : part);
            if (blockIdx.x == 0 && !stop)
                *p.norm = norm;
            const float f = p.max_norm / (norm + p.eps);
            s_factor = f < 1.f || f != f ? f : 1.f;
            s_stop = stop;
        }
    }
    if constexpr (!CLIP)
        return;
    __syncthreads();
    if (s_stop)
        return;
    const float factor = s_factor;
    // backwards: the tiles read last are still in L2
    if (tile == first)
        return;
    for (;;) {
        tile -= step;
        if (tile < t.tile0)
            seek(tile);
        base = (t.src & ~15ull) + static_cast<uint64_t>(tile - t.tile0) * kTileBytes;
        // in place, a factor of 1 changes nothing
        if (factor != 1.f || t.dst != t.src) {
            switch (t.types & 0xffu) {
            case CNS_DT_F32: rescale_tile<CNS_DT_F32>(t, base, end, factor); break;
            case CNS_DT_BF16: rescale_tile<CNS_DT_BF16>(t, base, end, factor); break;
            default: rescale_tile<CNS_DT_F16>(t, base, end, factor); break;
            }
        }
        if (tile < step)
            break;
    }
}

size_t workspace_bytes(int64_t count)
{
    return CNS_STEP_WORKSPACE_HEADER_BYTES + static_cast<size_t>(count) * sizeof(GradEntry);
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

// Tensors that the arguments have room for (32,764 bytes of them in all).
constexpr int kMostInline = 1000;

// Fill the table, in the arguments or the workspace, and launch.
template <int NORM, bool CLIP, int N>
int launch(const cns_grad_clip_t &g, const GradParams &p, const DeviceInfo &dev)
{
    cudaStream_t s = to_stream(g.stream);
    GradArgs<N> a;
    a.p = p;
    a.p.table = reinterpret_cast<const GradEntry *>(static_cast<char *>(g.workspace_dev) + CNS_STEP_WORKSPACE_HEADER_BYTES);
    a.p.count = 0;
    TableChunk c;
    c.n = 0;
    uint32_t tile0 = 0;
    for (int64_t i = 0; i < g.count; ++i) {
        const cns_tensor_t &t = g.grads[i];
        if (t.elems) {
            const cns_tensor_t &o = CLIP && g.outs ? g.outs[i] : t;
            const GradEntry e{reinterpret_cast<uint64_t>(t.data_dev), reinterpret_cast<uint64_t>(o.data_dev), t.elems,
                              tile0, static_cast<uint32_t>(t.dtype | o.dtype << 8)};
            tile0 += static_cast<uint32_t>(tiles_of(t));
            if constexpr (N > 0) {
                a.e[a.p.count++] = e;
            } else {
                c.e[c.n++] = e;
            }
        }
        if (N == 0 && (c.n == kChunkEntries || (c.n > 0 && i + 1 == g.count))) {
            c.to = const_cast<GradEntry *>(a.p.table) + a.p.count;
            grad_table_kernel<<<1, 128, 0, s>>>(c);
            CNS_CUDA(cudaGetLastError());
            a.p.count += c.n;
            c.n = 0;
        }
    }
    // one CTA an SM, fewer when there is not a tile for each
    const int most = std::min<int>(dev.sm_count, kStepMaxCtas);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::max(1, static_cast<int>(std::min<int64_t>(p.tiles, most))));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute coop;
    coop.id = cudaLaunchAttributeCooperative;
    coop.val.cooperative = 1;
    cfg.attrs = &coop;
    cfg.numAttrs = cfg.gridDim.x > 1 ? 1 : 0;
    void *args[] = {&a};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(grad_kernel<NORM, CLIP, N>), args);
    if (e == cudaErrorCooperativeLaunchTooLarge) {
        (void)cudaGetLastError();
        return CNS_ERR_NOT_RESIDENT;
    }
    return e == cudaSuccess ? CNS_SUCCESS : cuda_fail(e, "gradient launch");
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
    GradParams p = {};
    p.header = static_cast<uint32_t *>(g->workspace_dev);
    p.norm = g->norm_dev;
    p.timeout_ns = barrier_timeout_ns(g->timeout_ms);
    p.tiles = static_cast<uint32_t>(tiles);
    p.max_norm = g->max_norm;
    p.eps = g->eps;
    int rc;
    if (g->count <= 32)
        rc = g->norm_type == CNS_NORM_L2 ? launch<CNS_NORM_L2, CLIP, 32>(*g, p, dev) : launch<CNS_NORM_INF, CLIP, 32>(*g, p, dev);
    else if (g->count <= kMostInline)
        rc = g->norm_type == CNS_NORM_L2 ? launch<CNS_NORM_L2, CLIP, kMostInline>(*g, p, dev)
                                         : launch<CNS_NORM_INF, CLIP, kMostInline>(*g, p, dev);
    else
        rc = g->norm_type == CNS_NORM_L2 ? launch<CNS_NORM_L2, CLIP, 0>(*g, p, dev) : launch<CNS_NORM_INF, CLIP, 0>(*g, p, dev);
    if (rc)
        return rc;
    if (!g->sync)
        return CNS_SUCCESS;
    g->device_status = 0;
    if (int rc2 = syncall_read_workspace(g->workspace_dev, g->stream, nullptr, nullptr, &g->device_status))
        return rc2;
    return g->device_status;
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
