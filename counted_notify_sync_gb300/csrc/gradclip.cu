// gradclip.cu -- the global gradient norm over many tensors, and clipping by
// it (cns_grad_norm, cns_grad_clip).
//
//   norm = sqrt(sum over all tensors of x^2)   (or the largest |x|)
//   out  = x * min(1, max_norm / (norm + eps))
//
// One launch, one CTA an SM: read everything once and sum; then, for the norm
// alone, the last CTA joins the parts; to clip, the CTAs exchange them
// (step_device.cuh; a cooperative launch) and scale.
//
// Layout.  A tile is `vecs` 16-byte vectors a lane of one warp (512 B to 4 KB,
// all tiles of a call alike), cut at 16-byte boundaries of the address space:
// its vectors are aligned wherever its tensor starts, and only a tensor's
// first and last vector can be partial.  A round is one tile for each warp of
// the GPU, neighbours to a CTA, so that the rounds sweep through memory; `vecs`
// is chosen so that the last round is as full as the others.
//
// Bound.  The norm reads its bytes once: HBM (400M bf16 elements: 112.9 us, 7.1
// TB/s, 104 % of the measured copy rate).  Clipping has to read everything
// before it can write anything, so a set larger than the chip is read twice
// and written once: 400M bf16 to bf16 367 us, 6.5 TB/s over 2.4 GB.  What the
// chip holds it reads once:
//   - the last round stays in the registers it was summed from (20 MB over the
//     GPU) and the one before it in shared memory (20 MB);
//   - the three before those are loaded with an L2 evict-last hint (60 MB), all
//     others and all stores with evict-first, and the rounds are scaled
//     backwards.
// 25M f32 (100 MB in, 100 MB out): 54 us with neither, 47 us with all of this
// (50 us with streaming stores alone; 48 us without shared memory).  Keeping
// two rounds in shared memory instead (224 KB) took 54 us: loads in flight
// need L1, and too little of it was left.  Prefetching the lost rounds into L2
// while the CTAs exchange took 47 us.  Filling shared memory by bulk
// copies, which do not, was no faster at 3.5 KB a copy (46 us here, but the
// norm fell to 6.5 TB/s) and slower below: a bulk copy costs its SM some 50 ns.
// Small sets are a launch, a trip to memory and the join: the norm of 0.2M f32
// elements 3.9 us, in a loop as in a CUDA graph (by the exchange, which needs
// the cooperative launch, 6.2 and 4.5 us); clipping 1M elements 8.2 and 6.2 us.
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
constexpr int kRowBytes = 512;     // one 16-byte vector a lane
constexpr int kLaneVecs = 8;       // vectors of a lane in the largest tile
constexpr uint32_t kKeepL2 = 3;    // rounds that L2 is asked to keep, before the two that stay on the SM

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
    int32_t vecs;             // of a lane in a tile: the tile is vecs * kRowBytes
    float max_norm, eps;
    uint32_t start[kStepMaxCtas];   // the tensor that each CTA's first tile lies in
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
constexpr int kChunkEntries = 1000;   // 32 KB of arguments
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

// The tensor that `tile` lies in, between tensors lo and hi (tensors without
// elements have no tiles and are not in the table).
template <int N>
__device__ __forceinline__ int find_tensor(const GradArgs<N> &a, int lo, int hi, uint32_t tile)
{
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tile0_of(a, mid) <= tile)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// What L2 does with a line: kNormal as it likes; else a createpolicy value.
constexpr uint64_t kNormal = 0;

__device__ __forceinline__ uint64_t policy_evict_first()
{
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ uint64_t policy_evict_last()
{
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}

template <bool HINT>
__device__ __forceinline__ uint4 ld_stream(uint64_t a, uint64_t policy)
{
    uint4 v;
    if constexpr (HINT)
        asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(a), "l"(policy)
                     : "memory");
    else
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

// One tile: where it starts, where its first byte's value goes, and which of
// its bytes, lo .. len - 1, the tensor has.
struct Tile {
    uint64_t base, dst;
    int lo, len;
    uint32_t types;
};

// The calling lane's vectors of a tile.  A vector that the tensor covers only
// in part is loaded element by element; what it does not cover is 0.
template <int D>
__device__ __forceinline__ uint4 load_part(const Tile &t, int o)
{
    using T = typename Elem<D>::type;
    union { uint4 v; uint16_t h[8]; uint32_t w[4]; } u;
    u.v = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < Vec<D>::N; ++i) {
        const int at = o + i * static_cast<int>(sizeof(T));
        if (at >= t.lo && at < t.len) {
            if constexpr (sizeof(T) == 4)
                u.w[i] = *reinterpret_cast<const uint32_t *>(t.base + at);
            else
                u.h[i] = *reinterpret_cast<const uint16_t *>(t.base + at);
        }
    }
    return u.v;
}

template <int D, bool HINT>
__device__ __forceinline__ void load_tile(const Tile &t, int vecs, uint4 *v, uint64_t policy)
{
    const int mine = (threadIdx.x & 31u) * 16;
    if (t.lo == 0 && t.len == vecs * kRowBytes) {
#pragma unroll
        for (int j = 0; j < kLaneVecs; ++j)
            if (j < vecs)
                v[j] = ld_stream<HINT>(t.base + mine + j * kRowBytes, policy);
    } else {
#pragma unroll
        for (int j = 0; j < kLaneVecs; ++j) {
            const int o = mine + j * kRowBytes;
            if (j < vecs)
                v[j] = o >= t.lo && o + 16 <= t.len ? ld_stream<HINT>(t.base + o, policy) : load_part<D>(t, o);
        }
    }
}

// A tile's part of the norm for the calling lane: the sum of its squares, or
// its largest magnitude (as integers, so that NaN is above inf).
template <int NORM, int D>
__device__ __forceinline__ float tile_part(const uint4 *v, int vecs)
{
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kLaneVecs; ++j) {
        if (j >= vecs)
            break;
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

// A warp's part from its lanes'.
template <int NORM>
__device__ __forceinline__ float warp_part(float v)
{
    if constexpr (NORM == CNS_NORM_L2)
        return warp_sum(v);
    else
        return __uint_as_float(__reduce_max_sync(kFullWarp, __float_as_uint(v)));
}

// The norm from the CTAs' norms, r[i] that of CTA 32 i + lane (0 beyond the last).
template <int NORM>
__device__ __forceinline__ float joined(const float *r)
{
    uint32_t most = 0;
#pragma unroll
    for (uint32_t i = 0; i < kStepMaxCtas / 32; ++i)
        most = max(most, __float_as_uint(r[i]));
    float norm = __uint_as_float(__reduce_max_sync(kFullWarp, most));
    if (NORM == CNS_NORM_L2 && norm > 0.f && norm < INFINITY) {
        // squares of the largest one's parts: nothing overflows (a part is the root of a float: 2^-75 to 2^64)
        const float inverse = 1.f / norm;
        float sum = 0.f;
#pragma unroll
        for (uint32_t i = 0; i < kStepMaxCtas / 32; ++i) {
            const float y = r[i] * inverse;
            sum = fmaf(y, y, sum);
        }
        norm *= sqrtf(warp_sum(sum));
    }
    return norm;
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

// Store N (4 or 8) values in type D to an address that is a multiple of what
// they take there; they are not read again soon.
template <int D, int N>
__device__ __forceinline__ void store_aligned(uint64_t dst, const float *f)
{
    if constexpr (D == CNS_DT_F32 && N == 8)
        asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(f[0]), "f"(f[1]),
                     "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                     : "memory");
    else if constexpr (D == CNS_DT_F32)
        __stcs(reinterpret_cast<float4 *>(dst), make_float4(f[0], f[1], f[2], f[3]));
    else if constexpr (N == 8)
        __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(pack2<D>(f[0], f[1]), pack2<D>(f[2], f[3]),
                                                          pack2<D>(f[4], f[5]), pack2<D>(f[6], f[7])));
    else
        __stcs(reinterpret_cast<uint2 *>(dst), make_uint2(pack2<D>(f[0], f[1]), pack2<D>(f[2], f[3])));
}

// The same for values first .. last - 1 only, at any address of D's type.
template <int D, int N>
__device__ __forceinline__ void store_vec(uint64_t dst, const float *f, int first, int last)
{
    using T = typename Elem<D>::type;
    if (first == 0 && last == N && dst % (N * sizeof(T)) == 0) {
        store_aligned<D, N>(dst, f);
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i >= first && i < last)
            reinterpret_cast<T *>(dst)[i] = Elem<D>::put(f[i]);
}

template <int DS, int DD>
__device__ __forceinline__ void scale_tile(const Tile &t, int vecs, const uint4 *v, float factor)
{
    constexpr int S = static_cast<int>(sizeof(typename Elem<DS>::type));
    constexpr int T = static_cast<int>(sizeof(typename Elem<DD>::type));
    constexpr int N = Vec<DS>::N;
    const int mine = (threadIdx.x & 31u) * 16;
    const bool whole = t.lo == 0 && t.len == vecs * kRowBytes && t.dst % (N * T) == 0;
#pragma unroll
    for (int j = 0; j < kLaneVecs; ++j) {
        if (j >= vecs)
            break;
        const int o = mine + j * kRowBytes;
        float f[N];
        Vec<DS>::unpack(v[j], f);
#pragma unroll
        for (int i = 0; i < N; ++i)
            f[i] *= factor;
        if (whole) {
            store_aligned<DD, N>(t.dst + o / S * T, f);
        } else if (o + 16 > t.lo && o < t.len) {
            const int first = o < t.lo ? (t.lo - o) / S : 0;
            const int last = o + 16 > t.len ? (t.len - o) / S : N;
            store_vec<DD, N>(t.dst + o / S * T, f, first, last);
        }
    }
}

template <int D>
__device__ __forceinline__ void scale_into(const Tile &t, int vecs, const uint4 *v, float factor)
{
    switch (t.types >> 8) {
    case CNS_DT_F32: scale_tile<D, CNS_DT_F32>(t, vecs, v, factor); break;
    case CNS_DT_BF16: scale_tile<D, CNS_DT_BF16>(t, vecs, v, factor); break;
    default: scale_tile<D, CNS_DT_F16>(t, vecs, v, factor); break;
    }
}

template <int NORM, bool CLIP, int N>
__global__ void __launch_bounds__(kThreads, 1) grad_kernel(const __grid_constant__ GradArgs<N> a)
{
    const GradParams &p = a.p;
    extern __shared__ uint4 s_kept[];   // [vecs][kThreads], the last round but one
    __shared__ float s_part[kWarps];
    __shared__ float s_factor;
    __shared__ int s_stop;
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    // a round of tiles is one for each warp of the grid, neighbours to a CTA; the last one is shared out evenly
    const uint32_t full = kWarps * gridDim.x;
    const uint32_t rounds = (p.tiles + full - 1) / full;
    auto tile_of = [&](uint32_t round) {
        const uint32_t n = min(full, p.tiles - round * full);
        const uint32_t begin = n * blockIdx.x / gridDim.x, end = n * (blockIdx.x + 1) / gridDim.x;
        return begin + warp < end ? round * full + begin + warp : ~0u;
    };
    grid_dependency_wait();   // launched early: nothing of the tensors or the workspace before this
    uint32_t tag = 0;
    bool stop = false;
    if (warp == 0) {
        tag = ld_relaxed_gpu(p.header + kStepEpochWord) + 1u;
        stop = ld_relaxed_gpu(p.header + kStepStatusWord + 1) != 0u;   // an earlier call failed
    }

    uint4 v[kLaneVecs];
    int at = static_cast<int>(p.start[blockIdx.x]);
    uint32_t here = tile0_of(a, at);   // tensor `at` has the tiles here .. next - 1
    uint32_t next = at + 1 < p.count ? tile0_of(a, at + 1) : p.tiles;
    Tile tile{};
    auto visit = [&](uint32_t i) {
        if (i >= next || i < here) {
            // every tensor of the table has a tile, so it lies at most as many tensors away as tiles
            at = i >= next ? find_tensor(a, at + 1, static_cast<int>(min(p.count - 1u, at + (i - here))), i)
                           : find_tensor(a, at - static_cast<int>(min(static_cast<uint32_t>(at), here - i)), at - 1, i);
            here = tile0_of(a, at);
            next = at + 1 < p.count ? tile0_of(a, at + 1) : p.tiles;
        }
        const GradEntry t = entry_of(a, at);
        const int S = (t.types & 0xffu) == CNS_DT_F32 ? 4 : 2, T = (t.types >> 8) == CNS_DT_F32 ? 4 : 2;
        const int bytes = p.vecs * kRowBytes, ahead = static_cast<int>(t.src & 15u);
        // from the tensor's first element to the tile's first byte; before the tensor in its first tile
        const int64_t from = static_cast<int64_t>(i - here) * bytes - ahead;
        tile.types = t.types;
        tile.base = t.src + from;
        tile.dst = t.dst + from / S * T;
        tile.lo = i == here ? ahead : 0;
        tile.len = static_cast<int>(min(static_cast<int64_t>(bytes), t.elems * S - from));
    };
    auto load = [&](uint64_t policy) {
        switch (tile.types & 0xffu) {
        case CNS_DT_F32: load_tile<CNS_DT_F32, CLIP>(tile, p.vecs, v, policy); break;
        case CNS_DT_BF16: load_tile<CNS_DT_BF16, CLIP>(tile, p.vecs, v, policy); break;
        default: load_tile<CNS_DT_F16, CLIP>(tile, p.vecs, v, policy); break;
        }
    };
    const uint64_t fleeting = CLIP ? policy_evict_first() : kNormal, lasting = CLIP ? policy_evict_last() : kNormal;

    // a lane's sum over its tiles, 64 tiles at a time
    float part = 0.f, recent = 0.f;
    for (uint32_t round = 0; round < rounds; ++round) {
        const uint32_t i = tile_of(round);
        if (i == ~0u)
            continue;
        visit(i);
        const uint32_t left = rounds - 1 - round;
        load(left >= 2 && left < 2 + kKeepL2 ? lasting : fleeting);
        float f;
        switch (tile.types & 0xffu) {
        case CNS_DT_F32: f = tile_part<NORM, CNS_DT_F32>(v, p.vecs); break;
        case CNS_DT_BF16: f = tile_part<NORM, CNS_DT_BF16>(v, p.vecs); break;
        default: f = tile_part<NORM, CNS_DT_F16>(v, p.vecs); break;
        }
        if constexpr (NORM == CNS_NORM_L2) {
            recent += f;
            if ((round & 63u) == 63u) {
                part += recent;
                recent = 0.f;
            }
        } else {
            part = __uint_as_float(max(__float_as_uint(part), __float_as_uint(f)));
        }
        if (CLIP && left == 1) {
#pragma unroll
            for (int j = 0; j < kLaneVecs; ++j)
                if (j < p.vecs)
                    s_kept[j * kThreads + threadIdx.x] = v[j];
        }
    }
    part = warp_part<NORM>(NORM == CNS_NORM_L2 ? part + recent : part);
    if (lane == 0)
        s_part[warp] = part;
    __syncthreads();
    if (warp == 0) {
        // CTAs exchange roots: a sum of squares that is out of range for 32 bits may have a norm that is not
        part = warp_part<NORM>(s_part[lane]);
        float norm = NORM == CNS_NORM_L2 ? sqrtf(part) : part;
        float r[kStepMaxCtas / 32] = {};
        bool mine = blockIdx.x == 0;   // to write the norm
        if constexpr (CLIP) {
            if (gridDim.x > 1 && !stop) {
                send_all(p.header, gridDim.x, tag, __float_as_uint(norm));
                stop = receive_all(p.header, gridDim.x, tag, p.timeout_ns, r);
                norm = joined<NORM>(r);
                if (!stop && blockIdx.x == 0 && lane == 0)
                    st_relaxed_gpu(p.header + kStepEpochWord, tag);
            }
        } else if (gridDim.x > 1) {
            mine = gather_last(p.header, gridDim.x, __float_as_uint(norm), r);
            if (mine)
                norm = joined<NORM>(r);
        }
        if (lane == 0) {
            if (mine && !stop)
                *p.norm = norm;
            if constexpr (CLIP) {
                // inf / inf (no limit) and 0 / 0 clip nothing; NaN comes from a norm of NaN alone
                const float f = p.max_norm / (norm + p.eps);
                s_factor = f < 1.f || norm != norm ? f : 1.f;
                s_stop = stop;
            }
        }
    }
    if constexpr (!CLIP)
        return;
    __syncthreads();
    if (s_stop)
        return;
    const float factor = s_factor;
    // backwards: the last round is still in v, the one before it in shared memory, some before them in L2
    for (uint32_t left = 0; left < rounds; ++left) {
        const uint32_t i = tile_of(rounds - 1 - left);
        if (i == ~0u)
            continue;
        visit(i);
        if (factor == 1.f && tile.dst == tile.base)
            continue;   // in place, a factor of 1 changes nothing
        if (left == 1) {
#pragma unroll
            for (int j = 0; j < kLaneVecs; ++j)
                if (j < p.vecs)
                    v[j] = s_kept[j * kThreads + threadIdx.x];
        } else if (left > 1) {
            load(fleeting);
        }
        switch (tile.types & 0xffu) {
        case CNS_DT_F32: scale_into<CNS_DT_F32>(tile, p.vecs, v, factor); break;
        case CNS_DT_BF16: scale_into<CNS_DT_BF16>(tile, p.vecs, v, factor); break;
        default: scale_into<CNS_DT_F16>(tile, p.vecs, v, factor); break;
        }
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

// Bytes of the 16-byte vectors that a tensor touches, and its tiles.
int64_t span_of(const cns_tensor_t &t)
{
    const uint64_t a = reinterpret_cast<uint64_t>(t.data_dev);
    return static_cast<int64_t>(((a & 15u) + t.elems * elem_bytes(t.dtype) + 15) & ~15ull);
}

int64_t tiles_of(const cns_tensor_t &t, int vecs)
{
    const int64_t tile = vecs * kRowBytes;
    return t.elems ? (span_of(t) + tile - 1) / tile : 0;
}

// Tensors that the arguments have room for (32,764 bytes of them in all).
constexpr int kMostInline = 960;

// Fill the table, in the arguments or the workspace, and launch.
template <int NORM, bool CLIP, int N>
int launch(const cns_grad_clip_t &g, const GradParams &p, int ctas)
{
    cudaStream_t s = to_stream(g.stream);
    GradArgs<N> a;
    a.p = p;
    a.p.table = reinterpret_cast<const GradEntry *>(static_cast<char *>(g.workspace_dev) + CNS_STEP_WORKSPACE_HEADER_BYTES);
    a.p.count = 0;
    TableChunk c;
    c.n = 0;
    uint32_t tile0 = 0, cta = 0;
    const uint32_t first_round = std::min<uint32_t>(p.tiles, kWarps * ctas);
    for (int64_t i = 0; i < g.count; ++i) {
        const cns_tensor_t &t = g.grads[i];
        if (t.elems) {
            const cns_tensor_t &o = CLIP && g.outs ? g.outs[i] : t;
            const GradEntry e{reinterpret_cast<uint64_t>(t.data_dev), reinterpret_cast<uint64_t>(o.data_dev), t.elems,
                              tile0, static_cast<uint32_t>(t.dtype | o.dtype << 8)};
            tile0 += static_cast<uint32_t>(tiles_of(t, p.vecs));
            const int32_t index = a.p.count + c.n;
            // CTAs whose first tile lies in this tensor
            for (; cta < static_cast<uint32_t>(ctas) && first_round * cta / ctas < tile0; ++cta)
                a.p.start[cta] = static_cast<uint32_t>(index);
            if constexpr (N > 0)
                a.e[a.p.count++] = e;
            else
                c.e[c.n++] = e;
        }
        if (N == 0 && (c.n == kChunkEntries || (c.n > 0 && i + 1 == g.count))) {
            c.to = const_cast<GradEntry *>(a.p.table) + a.p.count;
            grad_table_kernel<<<1, 1024, 0, s>>>(c);
            CNS_CUDA(cudaGetLastError());
            a.p.count += c.n;
            c.n = 0;
        }
    }
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = CLIP && ctas > 1 ? together_launch(&attr) : early_launch(&attr);
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    if (CLIP && p.tiles > static_cast<uint32_t>(ctas) * kWarps) {   // more than one round
        cfg.dynamicSmemBytes = static_cast<size_t>(p.vecs) * kRowBytes * kWarps;
        CNS_CUDA(cudaFuncSetAttribute(grad_kernel<NORM, CLIP, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kLaneVecs * kRowBytes * kWarps));
    }
    void *args[] = {&a};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(grad_kernel<NORM, CLIP, N>), args);
    if (e == cudaErrorCooperativeLaunchTooLarge) {
        (void)cudaGetLastError();
        return CNS_ERR_NOT_RESIDENT;
    }
    return e == cudaSuccess ? CNS_SUCCESS : cuda_fail(e, "gradient launch");
}

template <int NORM, bool CLIP>
int launch_sized(const cns_grad_clip_t &g, const GradParams &p, int ctas)
{
    // the arguments are copied with each launch: no more room in them than it takes
    return g.count <= 64            ? launch<NORM, CLIP, 64>(g, p, ctas)
           : g.count <= kMostInline ? launch<NORM, CLIP, kMostInline>(g, p, ctas)
                                    : launch<NORM, CLIP, 0>(g, p, ctas);
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
    int64_t bytes = 0;
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
            bytes += span_of(g->grads[i]);
    }
    DeviceInfo dev;
    if (int rc = current_device(&dev))
        return rc;
    // tiles of equal size, so that every warp of the GPU takes the same number of them
    const int most = std::min<int>(dev.sm_count, kStepMaxCtas);
    const int64_t round = static_cast<int64_t>(most) * kWarps * kRowBytes;
    const int64_t rounds = (bytes + round * kLaneVecs - 1) / (round * kLaneVecs);
    GradParams p = {};
    p.vecs = rounds ? static_cast<int>((bytes + round * rounds - 1) / (round * rounds)) : 1;
    int64_t tiles = 0;
    for (int64_t i = 0; i < g->count; ++i)
        tiles += tiles_of(g->grads[i], p.vecs);
    if (tiles > 0x7fffffff)
        return CNS_ERR_INVALID_VALUE;
    p.header = static_cast<uint32_t *>(g->workspace_dev);
    p.norm = g->norm_dev;
    p.timeout_ns = barrier_timeout_ns(g->timeout_ms);
    p.tiles = static_cast<uint32_t>(tiles);
    p.max_norm = g->max_norm;
    p.eps = g->eps;
    // one CTA an SM, fewer when there is not a tile for each
    const int ctas = std::max(1, static_cast<int>(std::min<int64_t>(tiles, most)));
    if (int rc = g->norm_type == CNS_NORM_L2 ? launch_sized<CNS_NORM_L2, CLIP>(*g, p, ctas)
                                             : launch_sized<CNS_NORM_INF, CLIP>(*g, p, ctas))
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
