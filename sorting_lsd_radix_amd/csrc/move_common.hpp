// move_common.hpp -- parts of rows in registers, shared by the kernels that
// move rows by index (choices.hip, embed.hip).
#pragma once

#include "rows_common.hpp"

namespace rs {

constexpr int kMoveBlock = 256;
constexpr int kMoveWaves = kMoveBlock / kWave;

// Elements of a 16-byte vector.
template <class T>
constexpr int kVec = 16 / sizeof(T);

// The wave's number in its block, known to be the same for the whole wave.
__device__ __forceinline__ uint32_t wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); }

// The value of lane `from`, the same lane for the whole wave.
__device__ __forceinline__ uint32_t lane_value(uint32_t x, uint32_t from) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), static_cast<int>(from)));
}
__device__ __forceinline__ float lane_value(float x, uint32_t from) {
    return __uint_as_float(lane_value(__float_as_uint(x), from));
}

// A lane's U vectors of a row of at least one vector, 64 vectors apart.  The
// row's last vector begins where the row has a whole one left, so it may hold
// elements of the one before it: those are moved twice, with the same values.
template <class T, int U>
struct RowPart {
    static constexpr int V = kVec<T>;
    using Vec = AnyVec<16>::V;
    uint32_t at[U];     // first element
    bool real[U];       // whether the row has this vector

    __device__ __forceinline__ RowPart(uint32_t part, uint32_t width) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t c = ((part * U + u) * kWave + lane_id()) * V;
            real[u] = c < width;
            at[u] = c < width - V ? c : width - V;
        }
    }
    // Bits of vector u's elements that are its own, and not of the one before it
    // as well; none where the row has no such vector.
    __device__ __forceinline__ Vec own_bits(uint32_t part, int u) const {
        const uint32_t twice = real[u] ? ((part * U + u) * kWave + lane_id()) * V - at[u] : V;
        Vec m;
#pragma unroll
        for (uint32_t d = 0; d < 4; ++d) {
            if constexpr (sizeof(T) == 4) m[d] = d < twice ? 0u : ~0u;
            else m[d] = 2 * d + 1 < twice ? 0u : 2 * d < twice ? 0xFFFF0000u : ~0u;
        }
        return m;
    }
    // ONCE: past the caches, for what is too large to be found there again.  Lanes
    // behind the row's end read its last vector: without branches the loads go out together.
    template <bool ONCE = false>
    __device__ __forceinline__ void load(const T* row, Vec (&r)[U]) const {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Vec* from = reinterpret_cast<const Vec*>(row + at[u]);
            r[u] = ONCE ? __builtin_nontemporal_load(from) : *from;
        }
    }
    __device__ __forceinline__ void store(T* row, const Vec (&r)[U]) const {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (real[u]) *reinterpret_cast<Vec*>(row + at[u]) = r[u];
    }
};

// Waits for loaded registers here, so that reading them across lanes between the
// loads of rows does not wait for those (the rows of a piece of sorted tokens came
// one by one without it, 163 us against 134).
template <class A, class B>
__device__ __forceinline__ void arrived(A& a, B& b) {
    asm volatile("" : "+v"(a), "+v"(b));
}

// A vector's elements as f32, and back.
template <class T>
__device__ __forceinline__ void widen(AnyVec<16>::V r, float (&x)[kVec<T>]) {
    const auto e = __builtin_bit_cast(typename SomeVec<kVec<T>, T>::Elems, r);
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) x[j] = static_cast<float>(e.v[j]);
}
template <class T>
__device__ __forceinline__ AnyVec<16>::V narrow(const float (&x)[kVec<T>]) {
    typename SomeVec<kVec<T>, T>::Elems e;
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) e.v[j] = static_cast<T>(x[j]);
    return __builtin_bit_cast(AnyVec<16>::V, e);
}
// A vector times w, rounded.
template <class T>
__device__ __forceinline__ AnyVec<16>::V scaled(AnyVec<16>::V r, float w) {
    float x[kVec<T>];
    widen<T>(r, x);
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) x[j] *= w;
    return narrow<T>(x);
}

inline uint64_t up(uint64_t n, uint64_t d) { return (n + d - 1) / d; }

// Whether rows that are read once are read past the caches, which hold 256 MB on
// the package: combining a router's rows, others in between, takes at 64 MB 12.7 us
// by the caches and 13.4 past them, at 128 MB 28.9 and 26.8, at 512 MB 120 and 104;
// rows that the kernel before wrote take 33.0 and 33.5, 66.8 and 62.8, 293 and 272
// with that kernel.
inline bool large(uint64_t bytes) { return bytes > (uint64_t{96} << 20); }

// How rows are split among waves: vectors of a lane (1, 2 or 4, up to `most`, so
// many that the parts still fill the chip), and parts of a row.  By token, at most two:
// 32768 rows of 640 vectors 119 us with one, 91 with two, 95 with four; 100000 of 75 54.0, 41.5 and
// 41.3; 8192 of 512 17.4, 18.0 and 19.3.  To places, at most four: 16384 rows of 512 to 8 places each 303, 291
// and 281; 5000 of 1024 to 6 185, 165 and 166; 3001 of 251 to 5 13.1 each way.
struct Split {
    uint32_t unroll, parts;
};
inline Split split_rows(uint32_t vectors, uint64_t rows, uint32_t most) {
    const uint32_t each = (vectors + kWave - 1) / kWave;   // vectors of a lane, were a row one wave's
    uint32_t u = 1;
    while (u < most && u < each && rows * ((each + 2 * u - 1) / (2 * u)) >= 4096) u *= 2;
    return Split{u, (each + u - 1) / u};
}

}  // namespace rs
