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

// The value whose order pattern is `o` (a NaN for NaN's).
__device__ __forceinline__ float value_of_order32(uint32_t o) {
    return o == 1u ? __builtin_nanf("") : __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}

// Vectors of BYTES (a power of two up to 16) that may start on any element (2
// bytes, the smallest).  Named types, because copies by memcpy in two branches
// (whole and by element) are merged into loads and stores of single elements.
template <int BYTES>
struct AnyVec;
template <>
struct AnyVec<16> {
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct AnyVec<8> {
    typedef uint32_t V __attribute__((ext_vector_type(2), aligned(2)));
};
template <>
struct AnyVec<4> {
    typedef uint32_t V __attribute__((aligned(2)));
};
template <>
struct AnyVec<2> {
    typedef uint16_t V;
};

template <int V, class T>
struct SomeVec {
    static constexpr int kBytes = V * sizeof(T) < 16 ? V * sizeof(T) : 16;
    static constexpr int kParts = V * sizeof(T) / kBytes;
    static constexpr int kEach = V / kParts;
    using Part = typename AnyVec<kBytes>::V;
    struct Elems { T v[kEach]; };
};

// V consecutive elements at `at`, of which the first `n` exist; `fill` for the others.
template <int V, class T>
__device__ __forceinline__ void load_some(const T* at, uint32_t n, float fill, float (&x)[V]) {
    using S = SomeVec<V, T>;
    if (n >= V) {
        typename S::Part r[S::kParts];
#pragma unroll
        for (int p = 0; p < S::kParts; ++p) r[p] = *reinterpret_cast<const typename S::Part*>(at + p * S::kEach);
#pragma unroll
        for (int p = 0; p < S::kParts; ++p) {
            const auto e = __builtin_bit_cast(typename S::Elems, r[p]);
#pragma unroll
            for (int j = 0; j < S::kEach; ++j) x[p * S::kEach + j] = static_cast<float>(e.v[j]);
        }
    } else {
#pragma unroll
        for (uint32_t j = 0; j < V; ++j) x[j] = j < n ? static_cast<float>(at[j]) : fill;
    }
}

template <int V, class T>
__device__ __forceinline__ void store_some(T* at, uint32_t n, const float (&x)[V]) {
    using S = SomeVec<V, T>;
    if (n >= V) {
#pragma unroll
        for (int p = 0; p < S::kParts; ++p) {
            typename S::Elems e;
#pragma unroll
            for (int j = 0; j < S::kEach; ++j) e.v[j] = static_cast<T>(x[p * S::kEach + j]);
            *reinterpret_cast<typename S::Part*>(at + p * S::kEach) = __builtin_bit_cast(typename S::Part, e);
        }
    } else {
#pragma unroll
        for (uint32_t j = 0; j < V; ++j)
            if (j < n) at[j] = static_cast<T>(x[j]);
    }
}

// The value of lane ^ M, of any type of whole words.
template <int M, class T>
__device__ __forceinline__ T lane_xor_of(T x) {
    static_assert(sizeof(T) % 4 == 0, "whole words");
    uint32_t w[sizeof(T) / 4];
    __builtin_memcpy(w, &x, sizeof(T));
#pragma unroll
    for (uint32_t& v : w) v = lane_xor<M>(v);
    __builtin_memcpy(&x, w, sizeof(T));
    return x;
}

// op over aligned groups of N lanes; every lane of a group gets the result.
template <int N = kWave, class T, class Op>
__device__ __forceinline__ T lanes_reduce(T x, Op op) {
    if constexpr (N > 1) x = op(x, lane_xor_of<1>(x));
    if constexpr (N > 2) x = op(x, lane_xor_of<2>(x));
    if constexpr (N > 4) x = op(x, lane_xor_of<4>(x));
    if constexpr (N > 8) x = op(x, lane_xor_of<8>(x));
    if constexpr (N > 16) x = op(x, lane_xor_of<16>(x));
    if constexpr (N > 32) x = op(x, lane_xor_of<32>(x));
    return x;
}

template <int N = kWave, class T>
__device__ __forceinline__ T lanes_max(T x) {
    return lanes_reduce<N>(x, [](T a, T b) { return a > b ? a : b; });
}
template <int N = kWave>
__device__ __forceinline__ float lanes_max(float x) {
    return lanes_reduce<N>(x, [](float a, float b) { return fmaxf(a, b); });
}

template <int N = kWave>
__device__ __forceinline__ double lanes_max(double x) {
    return lanes_reduce<N>(x, [](double a, double b) { return fmax(a, b); });
}

template <int N = kWave, class T>
__device__ __forceinline__ T lanes_sum(T x) {
    return lanes_reduce<N>(x, [](T a, T b) { return a + b; });
}

// One step of a bitonic network over the wave's lanes: of lane and lane ^ J
// the lower keeps the larger where (lane & SIZE) == 0, the smaller elsewhere.
template <int SIZE, int J, class T>
__device__ __forceinline__ T lanes_merge_steps(T k, uint32_t lane) {
    const T o = lane_xor_of<J>(k);
    const bool keep_max = ((lane & J) == 0) == ((lane & SIZE) == 0);
    k = ((k > o) == keep_max) ? k : o;   // unsigned keys; of equal ones either will do
    if constexpr (J > 1) k = lanes_merge_steps<SIZE, J / 2>(k, lane);
    return k;
}

// The keys of every aligned group of N lanes in decreasing order.
template <int N, int SIZE = 2, class T>
__device__ __forceinline__ T lanes_sort_desc(T k) {
    if constexpr (N > 1) k = lanes_merge_steps<SIZE, SIZE / 2>(k, lane_id() & (N - 1));
    if constexpr (SIZE < N) k = lanes_sort_desc<N, SIZE * 2>(k);
    return k;
}

template <class T>
__device__ __forceinline__ T wave_sort_desc(T k) {
    return lanes_sort_desc<kWave>(k);
}

// The best 64 of two lists in decreasing order, in decreasing order: the
// larger of lane l of one and lane 63 - l of the other form a bitonic sequence.
template <class T>
__device__ __forceinline__ T wave_merge_desc(T x, T y) {
    T r = lane_xor_of<1>(y);
    r = lane_xor_of<2>(r);
    r = lane_xor_of<4>(r);
    r = lane_xor_of<8>(r);
    r = lane_xor_of<16>(r);
    r = lane_xor_of<32>(r);
    return lanes_merge_steps<kWave, kWave / 2>(x > r ? x : r, lane_id());
}

}  // namespace rs
