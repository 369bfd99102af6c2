// Element access and row reductions of the row-wise operators
// (layer_norm.hip, int8_quant.hip, adamw_multi.hip): vectors of 16 bytes at
// any element alignment (gfx950 loads and stores dwords at any byte address;
// the operators take rows of any length and stride), bf16 or fp32 widened to
// fp32 exactly and rounded to nearest even once on the way out.
#pragma once

#include <type_traits>

#include "fp8q_device.h"

namespace fp8q {

// elements of T in 16 bytes
template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));     // at any element address

template <typename T>
__device__ __forceinline__ u32x4 load16(const T* p)
{
    return *reinterpret_cast<const u32x4_any*>(p);
}

template <typename T>
__device__ __forceinline__ void store16(T* p, u32x4 v)
{
    *reinterpret_cast<u32x4_any*>(p) = v;
}

// one element as fp32, and back (uint16_t: bf16 bits)
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return (float)__builtin_bit_cast(__bf16, x); }

template <typename T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ float narrow<float>(float x) { return x; }
template <> __device__ __forceinline__ uint16_t narrow<uint16_t>(float x)
{
    return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// the elements of 16 loaded bytes
template <typename T>
__device__ __forceinline__ void unpack(u32x4 w, float* v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        } else {
            v[i] = __uint_as_float(w[i]);
        }
    }
}

template <typename T>
__device__ __forceinline__ u32x4 pack(const float* v)
{
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2)
            w[i] = (uint32_t)narrow<uint16_t>(v[2 * i]) | (uint32_t)narrow<uint16_t>(v[2 * i + 1]) << 16;
        else
            w[i] = __float_as_uint(v[i]);
    }
    return w;
}

// Elements [c, c + kVec) of a row of `cols`; those at or past `cols` read as
// zero (no byte past the row's last element is touched).
template <typename T>
__device__ __forceinline__ u32x4 load_row(const T* row, int64_t c, int64_t cols)
{
    if (c + kVec<T> <= cols) return load16(row + c);
    u32x4 w = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) {
        if (c + i >= cols) break;
        if constexpr (sizeof(T) == 2) w[i / 2] |= (uint32_t)row[c + i] << (16 * (i & 1));
        else w[i] = __float_as_uint(row[c + i]);
    }
    return w;
}

template <typename T>
__device__ __forceinline__ void store_row(T* row, int64_t c, int64_t cols, u32x4 w)
{
    if (c + kVec<T> <= cols) {
        store16(row + c, w);
        return;
    }
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) {
        if (c + i >= cols) break;
        if constexpr (sizeof(T) == 2) row[c + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        else row[c + i] = __uint_as_float(w[i]);
    }
}

// Sum and maximum over the 64 lanes of a wave, in every lane (all active):
// four steps within the rows of 16 lanes as data-parallel moves, then the row
// and half-wave swaps, each of which leaves a lane its own value and its
// partner's (no trip through LDS; the tree is the same for every lane).
template <typename Op>
__device__ __forceinline__ float wave_reduce(float v, Op op)
{
    auto step = [&](auto ctrl) {
        return op(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF,
                                                                false)));
    };
    v = step(std::integral_constant<int, 0xB1>{});    // quad [1,0,3,2]
    v = step(std::integral_constant<int, 0x4E>{});    // quad [2,3,0,1]
    v = step(std::integral_constant<int, 0x141>{});   // half-row mirror
    v = step(std::integral_constant<int, 0x140>{});   // row mirror
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
    const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return op(__uint_as_float(h[0]), __uint_as_float(h[1]));
}

__device__ __forceinline__ float wave_sum(float v)
{
    return wave_reduce(v, [](float a, float b) { return a + b; });
}

__device__ __forceinline__ float wave_max(float v)
{
    return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace fp8q
