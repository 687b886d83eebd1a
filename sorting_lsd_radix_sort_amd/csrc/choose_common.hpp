// choose_common.hpp -- what the kernels of a router's choice and of beam search share:
// order keys of values, reductions over the lanes that serve a row together.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "row_vectors.hpp"

namespace lrs_choose {

using namespace lrs_rows;

// ---------------------------------------------------------------- order keys
//
// Unsigned integers in the order of the values: 0 for -infinity (nothing to choose), the
// largest for NaN, one key for both zeros.
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
    const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return v == -__builtin_inff() ? 0u : v != v ? ~0u : k;
}

__device__ __forceinline__ uint64_t key_of(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    const uint64_t k = b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
    return v == -__builtin_inf() ? 0ull : v != v ? ~0ull : k;
}

// The value of a key: -infinity for 0, NaN for the largest.
__device__ __forceinline__ float value_of(uint32_t k)
{
    const float v = __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
    return k == 0u ? -__builtin_inff() : v;
}

__device__ __forceinline__ double value_of(uint64_t k)
{
    const double v = __builtin_bit_cast(double, k & 0x8000000000000000ull ? k ^ 0x8000000000000000ull : ~k);
    return k == 0ull ? -__builtin_inf() : v;
}

// --------------------------------------------------------------------- teams
//
// Reductions over the L lanes of a team, given to all of them: lanes 1 and 2 apart by
// quad permutations, 4 and 8 by mirrors of half rows and rows (whose lanes hold the
// same by then), rows of 16 and halves by exchanging them between two copies.  Sums have
// one order whatever the lane.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

template <int L, typename F>
__device__ __forceinline__ uint32_t team_reduce(uint32_t v, F &&f)
{
    v = f(v, dpp<0xB1>(v));
    v = f(v, dpp<0x4E>(v));
    v = f(v, dpp<0x141>(v));
    if constexpr (L >= 16) v = f(v, dpp<0x140>(v));
    if constexpr (L >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = f((uint32_t)r[0], (uint32_t)r[1]);
    }
    if constexpr (L == 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = f((uint32_t)r[0], (uint32_t)r[1]);
    }
    return v;
}

template <int L>
__device__ __forceinline__ uint32_t team_max(uint32_t v)
{
    return team_reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

template <int L>
__device__ __forceinline__ uint32_t team_min(uint32_t v)
{
    return team_reduce<L>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

template <int L>
__device__ __forceinline__ uint32_t team_or(uint32_t v)
{
    return team_reduce<L>(v, [](uint32_t a, uint32_t b) { return a | b; });
}

template <int L>
__device__ __forceinline__ float team_sum(float v)
{
    return __builtin_bit_cast(float, team_reduce<L>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    }));
}

// Of two floats the larger, passing over NaN.
template <int L>
__device__ __forceinline__ float team_maxf(float v)
{
    return __builtin_bit_cast(float, team_reduce<L>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
    }));
}

template <int L>
__device__ __forceinline__ uint64_t team_max64(uint64_t v)
{
#pragma unroll
    for (int d = 1; d < L; d *= 2) {
        const uint64_t o = __shfl_xor((unsigned long long)v, d, L);
        v = o > v ? o : v;
    }
    return v;
}

template <int L>
__device__ __forceinline__ double team_sum64(double v)
{
#pragma unroll
    for (int d = 1; d < L; d *= 2) v += __shfl_xor(v, d, L);
    return v;
}

// What a lane stored to LDS before this is there for the others of its wave after it.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace lrs_choose
