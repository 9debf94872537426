// Device helpers shared by the mixer kernels (head norms with rotation, slot selection, the gated
// linear recurrence): element types, their conversions, and lane exchanges of the 64-wide wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sdm_device.hpp"

namespace sdm {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// A bfloat16 element in memory. Widening is exact; narrowing rounds once, to nearest even.
struct bf16_t {
    uint16_t bits;
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(bf16_t x) { return bf16_bits_to_f32(x.bits); }

template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ bf16_t narrow<bf16_t>(float x) { return bf16_t{__builtin_bit_cast(uint16_t, static_cast<__bf16>(x))}; }

// Two floats rounded to a word of two bfloat16 (one instruction on gfx950).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef float f32x2_ __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_{lo, hi}, bf16x2));
}

// The value of lane (lane ^ M), M a power of two: cross-lane moves inside the vector unit where the
// architecture has one (quads, rows of 16, the gfx950 swaps of rows and of halves), else the swizzle.
template <int M>
__device__ __forceinline__ uint32_t lane_xor(uint32_t x) {
    static_assert(M == 1 || M == 2 || M == 4 || M == 8 || M == 16 || M == 32, "a power of two below 64");
    if constexpr (M == 1) {
        return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xF, 0xF, true));   // quad_perm 1,0,3,2
    } else if constexpr (M == 2) {
        return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xF, 0xF, true));   // quad_perm 2,3,0,1
    } else if constexpr (M == 4) {
        return static_cast<uint32_t>(__builtin_amdgcn_ds_swizzle(static_cast<int>(x), (4 << 10) | 0x1F));
    } else if constexpr (M == 8) {
        return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x128, 0xF, 0xF, true));  // row_ror:8
    } else if constexpr (M == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        return (lane_id() & 16) ? r[0] : r[1];
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        return (lane_id() & 32) ? r[0] : r[1];
    }
}

template <int M>
__device__ __forceinline__ float lane_xor_f(float x) { return __uint_as_float(lane_xor<M>(__float_as_uint(x))); }

// The sum over each aligned group of G lanes, in every lane of it (a fixed tree).
template <int G>
__device__ __forceinline__ float group_sum(float x) {
    if constexpr (G >= 2) x += lane_xor_f<1>(x);
    if constexpr (G >= 4) x += lane_xor_f<2>(x);
    if constexpr (G >= 8) x += lane_xor_f<4>(x);
    if constexpr (G >= 16) x += lane_xor_f<8>(x);
    if constexpr (G >= 32) x += lane_xor_f<16>(x);
    if constexpr (G >= 64) x += lane_xor_f<32>(x);
    return x;
}

}  // namespace sdm
