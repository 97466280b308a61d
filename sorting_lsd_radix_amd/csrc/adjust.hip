// adjust.hip -- penalties of repeated tokens, biases and grammar masks on rows
// of logits, in one pass.
//
// A block takes a slice of a row's vocabulary.  Its logits and mask bits are on
// their way to registers while the block keeps a word for each token of the slice
// in LDS and marks there what the row's lists say of the slice's tokens: the last
// bias entry that names one, how often one occurs behind the prompt, whether in
// the prompt.  The marks are maxima, sums and bits, so the order of the atomics does
// not matter.  Every block of a row reads the row's whole lists, from the caches.
#include <type_traits>

#include "internal.hpp"
#include "move_common.hpp"

namespace rs {

namespace {

#ifndef AB
#define AB 512
#endif
constexpr int kAdjustBlock = AB;

// A token's word: from the low end a bias entry's index + 1, the occurrences
// behind the prompt, a bit for an occurrence in it.
template <class W>
struct Word {
    static constexpr int kEntryBits = 0, kCountBits = 0;
};
template <>
struct Word<uint32_t> {
    static constexpr int kEntryBits = 16, kCountBits = 15;
};
template <>
struct Word<unsigned long long> {
    static constexpr int kEntryBits = 31, kCountBits = 32;
};
struct NoWord {};

// What a row's lists hold, each count within its list.
__device__ __forceinline__ uint32_t within(const int32_t* n, uint32_t r, uint32_t otherwise, uint32_t all) {
    if (n == nullptr) return otherwise;
    const int32_t x = n[r];
    return x < 0 ? 0u : static_cast<uint32_t>(x) < all ? static_cast<uint32_t>(x) : all;
}

constexpr int kTokens = 4;   // of a vector load
constexpr int kAhead = 2;    // vectors of history in flight
typedef uint32_t Tokens __attribute__((ext_vector_type(kTokens), aligned(4)));

// Tokens i .. i + 4 of `length`; what is behind them is no token.
__device__ __forceinline__ Tokens load_tokens(const uint32_t* from, uint32_t i, uint32_t length) {
    Tokens v = {~0u, ~0u, ~0u, ~0u};
    if (i + kTokens <= length) return *reinterpret_cast<const Tokens*>(from + i);
#pragma unroll
    for (int j = 0; j < kTokens; ++j)
        if (i + j < length) v[j] = from[i + j];
    return v;
}

// HOLD vectors a thread.  W: a token's word, or NoWord without lists.
template <class T, class O, class W, int HOLD>
__global__ __launch_bounds__(kAdjustBlock) void adjust_kernel(AdjustArgs a, uint32_t slices) {
    constexpr int V = kVec<T>;
    constexpr bool LISTS = !std::is_same<W, NoWord>::value;
    constexpr uint32_t kSlice = kAdjustBlock * HOLD * V;
    using Vec = AnyVec<16>::V;
    const uint32_t b = block_id(), tid = threadIdx.x;
    const uint32_t r = b / slices;
    if (r >= a.rows) return;
    const uint32_t lo = b % slices * kSlice;
    const uint32_t size = a.vocab - lo < kSlice ? a.vocab - lo : kSlice;
    const T* from = static_cast<const T*>(a.logits) + r * a.row_stride + lo;
    O* to = static_cast<O*>(a.out) + r * a.out_stride + lo;
    const uint32_t* mask = a.mask + r * a.mask_stride + lo / 32;

    Vec x[HOLD];
    uint32_t allowed[HOLD];
#pragma unroll
    for (int h = 0; h < HOLD; ++h) {
        const uint32_t i = (h * kAdjustBlock + tid) * V;
        allowed[h] = a.mask && i < size ? mask[i / 32] >> (i % 32) : ~0u;
        if (i + V <= size) {
            x[h] = *reinterpret_cast<const Vec*>(from + i);
        } else {
            float e[V];
            load_some<V>(from + i, i < size ? size - i : 0u, 0.0f, e);
            x[h] = narrow<T>(e);   // exact: they are T's
        }
    }

    float by = 1.0f, frequency = 0.0f, presence = 0.0f;
    __shared__ typename std::conditional<LISTS, W, char>::type s_word[LISTS ? kSlice : 1];
    if constexpr (LISTS) {
        constexpr W kOne = W{1} << Word<W>::kEntryBits;
        constexpr W kPrompt = kOne << Word<W>::kCountBits;
        const uint32_t length = a.history ? within(a.lengths, r, a.history_len, a.history_len) : 0u;
        const uint32_t prompt = within(a.prompt_lengths, r, 0u, length);
        const uint32_t* history = a.history + r * a.history_stride;
        constexpr uint32_t kRound = kAdjustBlock * kTokens * kAhead;
        Tokens next[kAhead];
        auto load = [&](uint32_t i0) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) next[k] = load_tokens(history, i0 + (k * kAdjustBlock + tid) * kTokens, length);
        };
        load(0);
        if (length > 0) {
            if (a.repetition) by = a.repetition[r];
            if (a.frequency) frequency = a.frequency[r];
            if (a.presence) presence = a.presence[r];
        }
#pragma unroll
        for (uint32_t i = 0; i < kSlice / kAdjustBlock; i += 16 / sizeof(W)) {
            typedef W Zero __attribute__((ext_vector_type(16 / sizeof(W))));
            *reinterpret_cast<Zero*>(&s_word[i * kAdjustBlock + tid * (16 / sizeof(W))]) = Zero{};
        }
        __syncthreads();
        if (a.bias_ids) {
            for (uint32_t i = tid; i < a.bias_len; i += kAdjustBlock) {
                const uint32_t v = a.bias_ids[r * a.bias_ids_stride + i] - lo;
                if (v < size) atomicMax(&s_word[v], static_cast<W>(i + 1));
            }
            __syncthreads();
        }
        for (uint32_t i0 = 0; i0 < length; i0 += kRound) {
            Tokens now[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) now[k] = next[k];
            if (i0 + kRound < length) load(i0 + kRound);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const uint32_t i = i0 + (k * kAdjustBlock + tid) * kTokens;
#pragma unroll
                for (int j = 0; j < kTokens; ++j) {
                    const uint32_t v = now[k][j] - lo;   // a token that is none lies behind every slice
                    if (v >= size) continue;
                    if (i + j < prompt) atomicOr(&s_word[v], kPrompt);
                    else atomicAdd(&s_word[v], kOne);
                }
            }
        }
        __syncthreads();
    }

#pragma unroll
    for (int h = 0; h < HOLD; ++h) {
        const uint32_t i = (h * kAdjustBlock + tid) * V;
        if (i >= size) break;
        float l[V];
        widen<T>(x[h], l);
        if constexpr (LISTS) {
            constexpr W kOne = W{1} << Word<W>::kEntryBits;
            constexpr W kPrompt = kOne << Word<W>::kCountBits;
            W w[V], any = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                w[j] = s_word[i + j];
                any |= w[j];
            }
            if (any != 0) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const uint32_t count = static_cast<uint32_t>((w[j] & (kPrompt - 1)) >> Word<W>::kEntryBits);
                    const uint32_t entry = static_cast<uint32_t>(w[j] & (kOne - 1));
                    if (w[j] >= kOne) l[j] = l[j] > 0.0f ? l[j] / by : l[j] * by;
                    if (count > 0) l[j] -= fmaf(frequency, static_cast<float>(count), presence);
                    if (entry > 0) l[j] += a.bias[r * a.bias_stride + entry - 1];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = (allowed[h] >> j) & 1u ? l[j] : -__builtin_huge_valf();
        store_some<V>(to + i, size - i, l);
    }
}

template <class T, class O, class W, int HOLD>
void launch_as(const AdjustArgs& a, hipStream_t stream) {
    constexpr uint32_t kSlice = kAdjustBlock * HOLD * kVec<T>;
    const uint32_t slices = (a.vocab + kSlice - 1) / kSlice;
    adjust_kernel<T, O, W, HOLD><<<many_blocks(static_cast<uint64_t>(a.rows) * slices), kAdjustBlock, 0, stream>>>(a, slices);
}

#ifndef HT
#define HT 1024
#endif
template <class T, class O>
hipError_t adjust_of(const AdjustArgs& a, hipStream_t stream) {
    // the fields of a wide word only where the lists can be longer than a narrow one's
    const bool wide = a.history_len >= (1u << Word<uint32_t>::kCountBits) || a.bias_len >= (1u << Word<uint32_t>::kEntryBits);
    const bool lists = a.history || a.bias_ids;
    // vectors a thread: as many as leave the chip enough blocks
    const uint64_t vectors = static_cast<uint64_t>(a.rows) * ((a.vocab + kVec<T> - 1) / kVec<T>);
    const int hold = vectors >= uint64_t{4} * HT * kAdjustBlock ? 4 : vectors >= uint64_t{2} * HT * kAdjustBlock ? 2 : 1;
    timing_before(stream, RS_KERNEL_ADJUST);
    if (!lists) {
        if (hold == 1) launch_as<T, O, NoWord, 1>(a, stream);
        else if (hold == 2) launch_as<T, O, NoWord, 2>(a, stream);
        else launch_as<T, O, NoWord, 4>(a, stream);
    } else if (wide) {
        if (hold == 1) launch_as<T, O, unsigned long long, 1>(a, stream);
        else launch_as<T, O, unsigned long long, 2>(a, stream);
    } else {
        if (hold == 1) launch_as<T, O, uint32_t, 1>(a, stream);
        else if (hold == 2) launch_as<T, O, uint32_t, 2>(a, stream);
        else launch_as<T, O, uint32_t, 4>(a, stream);
    }
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

}  // namespace

hipError_t launch_adjust(int elem_type, int out_type, const AdjustArgs& a, hipStream_t stream) {
    const bool f32 = out_type == RS_ELEM_F32;
    switch (elem_type) {
        case RS_ELEM_F32: return adjust_of<float, float>(a, stream);
        case RS_ELEM_F16: return f32 ? adjust_of<_Float16, float>(a, stream) : adjust_of<_Float16, _Float16>(a, stream);
        default: return f32 ? adjust_of<__bf16, float>(a, stream) : adjust_of<__bf16, __bf16>(a, stream);
    }
}

}  // namespace rs
