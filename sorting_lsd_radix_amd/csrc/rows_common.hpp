// rows_common.hpp -- loads, stores, order patterns and wave reductions shared
// by the kernels on rows of scores (route.hip, logprobs.hip).
#pragma once

#include "device_common.hpp"

namespace rs {

// A launch of many independent blocks: a grid dimension holds less than 2^32
// work items, so more than 2^16 blocks take two.  Blocks behind the last one
// return at once.
inline dim3 many_blocks(uint64_t blocks) {
    constexpr uint64_t kX = 1u << 16;
    return blocks <= kX ? dim3(static_cast<uint32_t>(blocks))
                        : dim3(static_cast<uint32_t>(kX), static_cast<uint32_t>((blocks + kX - 1) / kX));
}

__device__ __forceinline__ uint32_t block_id() { return blockIdx.y * gridDim.x + blockIdx.x; }

// Storage types of a matrix's elements, by rs_elem_type.
template <int ELEM>
struct Elem;
template <>
struct Elem<RS_ELEM_F32> {
    using T = float;
};
template <>
struct Elem<RS_ELEM_F16> {
    using T = _Float16;
};
template <>
struct Elem<RS_ELEM_BF16> {
    using T = __bf16;
};

// Order pattern of a score: unsigned order is the order within a row (larger
// values larger, -0.0 equal to +0.0, NaN below -inf), and no pattern is 0, so
// that 0 stands for "no element".
__device__ __forceinline__ uint32_t order32(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);   // -0.0 becomes +0.0
    const uint32_t sign = static_cast<uint32_t>(static_cast<int32_t>(u) >> 31);
    return (x == x) ? u ^ (sign | 0x80000000u) : 1u;
}

// The same in 64 bits, for scores that are compared in 64 bits; -inf and NaN
// (masked) share one pattern, 1.
__device__ __forceinline__ uint64_t order64_masked(double x) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
    const uint64_t sign = static_cast<uint64_t>(static_cast<int64_t>(u) >> 63);
    return (x > -__builtin_huge_val()) ? u ^ (sign | 0x8000000000000000ull) : 1ull;
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor(x, off, kWave));
    return x;
}

template <class T>
__device__ __forceinline__ T wave_sum(T x) {
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) x += __shfl_xor(x, off, kWave);
    return x;
}

}  // namespace rs
