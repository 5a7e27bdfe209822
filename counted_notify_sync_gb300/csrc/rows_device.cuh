// rows_device.cuh -- what the operators on rows (expert_rows.cu, rms_norm*.cu)
// share: accesses of 1 to 16 bytes and their elements in 32 bits.
#pragma once

#include <cstdint>

#include "step_device.cuh"

namespace cns {

// An access of A bytes.
template <int A> struct Bits;
template <> struct Bits<16> { using type = uint4; };
template <> struct Bits<8> { using type = uint2; };
template <> struct Bits<4> { using type = uint32_t; };
template <> struct Bits<2> { using type = uint16_t; };
template <> struct Bits<1> { using type = uint8_t; };

// The elements of an access, in 32 bits, and back (rounded to the nearest).
template <int D, int A>
__device__ __forceinline__ void unpack(const typename Bits<A>::type &raw, float *v)
{
    using T = typename Elem<D>::type;
    const T *e = reinterpret_cast<const T *>(&raw);
#pragma unroll
    for (int i = 0; i < A / static_cast<int>(sizeof(T)); ++i)
        v[i] = Elem<D>::get(e[i]);
}

template <int D, int A>
__device__ __forceinline__ typename Bits<A>::type pack(const float *v)
{
    using T = typename Elem<D>::type;
    constexpr int N = A / static_cast<int>(sizeof(T));
    typename Bits<A>::type raw;
    if constexpr (N % 2 == 0 && D == CNS_DT_BF16) {   // two at a time: one instruction
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            reinterpret_cast<__nv_bfloat162 *>(&raw)[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    } else if constexpr (N % 2 == 0 && D == CNS_DT_F16) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            reinterpret_cast<__half2 *>(&raw)[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    } else {
        T *e = reinterpret_cast<T *>(&raw);
#pragma unroll
        for (int i = 0; i < N; ++i)
            e[i] = Elem<D>::put(v[i]);
    }
    return raw;
}

// The widest access that all of `bits` (addresses, strides and lengths in bytes, or-ed together) are multiples of.
inline int access_bytes(uint64_t bits)
{
    for (int a = 16; a > 1; a /= 2)
        if (bits % a == 0)
            return a;
    return 1;
}

inline uint64_t address(const void *p) { return reinterpret_cast<uintptr_t>(p); }

}  // namespace cns
