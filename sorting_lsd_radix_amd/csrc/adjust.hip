// adjust.hip -- penalties of repeated tokens, biases and grammar masks on rows
// of logits, in one pass.
//
// A block takes a slice of a row's vocabulary.  Its logits, mask bits and the first
// of the row's tokens are on their way to registers while the block clears a mark
// for each token of the slice in LDS.  There it counts how often one occurs behind
// the prompt and notes whether one occurs in it or has a bias, which a table of the
// slice's biased tokens holds, the last entry's of each.  Marks are sums, bits and
// maxima, so the order of the atomics does not matter.  Every block of a row reads
// the row's whole lists, from the caches.
//
// What bounds it: 256 rows of 131072 bf16 take 25 us without lists (5.3 TB/s), 26 with
// histories of up to 500 tokens, 42 with up to 8192 and 300 biases, where the marking's
// instructions and atomics keep the VALU two thirds busy.
#include <type_traits>

#include "internal.hpp"
#include "move_common.hpp"

namespace rs {

namespace {

constexpr int kAdjustBlock = 512;

// What a block keeps of its tokens: nothing without lists; 16 bits for short
// histories, 32 for long ones, with a bit for an occurrence in the prompt, one for
// a bias, whose entry is then looked up, and the occurrences behind the prompt; 64
// for many biases, with the prompt's bit, the occurrences (32 bits) and a bias
// entry's index + 1 (31 bits).
enum Marks { kNoMarks, kMarks16, kMarks32, kMarks64 };
constexpr uint32_t kMaxHistory16 = 1u << 14;
constexpr uint32_t kMaxLooked = kAdjustBlock;   // bias entries that are looked up
constexpr uint32_t kSlots = 2 * kMaxLooked;     // of their table: a token is in the first free one from its low bits on
constexpr uint32_t kFree = ~0u;

// What a row's lists hold, each count within its list.
__device__ __forceinline__ uint32_t within(const int32_t* n, uint32_t r, uint32_t otherwise, uint32_t all) {
    if (n == nullptr) return otherwise;
    const int32_t x = n[r];
    return x < 0 ? 0u : static_cast<uint32_t>(x) < all ? static_cast<uint32_t>(x) : all;
}

constexpr int kTokens = 4;   // of a vector load
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

// HOLD vectors a thread.
template <class T, class O, Marks MARKS, int HOLD>
__global__ __launch_bounds__(kAdjustBlock) void adjust_kernel(AdjustArgs a, uint32_t slices) {
    constexpr int V = kVec<T>;
    constexpr uint32_t kSlice = kAdjustBlock * HOLD * V;
    constexpr bool kLooked = MARKS == kMarks16 || MARKS == kMarks32;
    using Vec = AnyVec<16>::V;
    typedef unsigned long long Word;
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

    constexpr uint32_t kBits = MARKS == kMarks16 ? 16 : MARKS == kMarks32 ? 32 : 64;
    constexpr uint32_t kVectors = MARKS == kNoMarks ? 1 : kSlice * kBits / 128;
    __shared__ u32x4 s_marks[kVectors];
    uint32_t* s_mark = reinterpret_cast<uint32_t*>(s_marks);   // 16 bits: of two tokens
    Word* s_word = reinterpret_cast<Word*>(s_marks);           // 64 bits
    constexpr Word kOne = Word{1} << 31, kPrompt64 = Word{1} << 63;
    constexpr uint32_t kPrompt = 1u << (kBits % 64 - 1) % 32, kBiased = kPrompt >> 1;
    __shared__ uint32_t s_token[kLooked ? kSlots : 1], s_entry[kLooked ? kSlots : 1];
    __shared__ float s_bias[kLooked ? kSlots : 1];
    // A division is a product with the inverse and what that leaves times the inverse
    // again: off by half a step and 2^-22 of one at most, for logits from 2^-100 on (below,
    // by two steps at most).  Where that is NaN, l is divided: for what is infinite, and for
    // penalties whose inverse may be inexact, infinite or 0, which is NaN itself.  (The product
    // alone, 1.5 steps: 256 rows of 131072 with histories up to 8192 41.6 us for 42.2.)
    float by = 1.0f, inverse = 1.0f, frequency = 0.0f, presence = 0.0f;
    // a logit of a token that the history holds `count` times behind the prompt
    auto penalised = [&](float l, bool seen, uint32_t count) {
        const bool up = l > 0.0f;
        float scaled = l * (up ? inverse : by);
        if (up) {
            scaled = fmaf(fmaf(-scaled, by, l), inverse, scaled);
            if (scaled != scaled) scaled = l / by;
        }
        if (seen) l = scaled;
        return l - (count > 0 ? fmaf(frequency, static_cast<float>(count), presence) : 0.0f);
    };
    if constexpr (MARKS != kNoMarks) {
        const uint32_t* history = a.history + r * a.history_stride;
        constexpr uint32_t kRound = kAdjustBlock * kTokens;
        // a round ahead, the first before the length is known
        Tokens next = load_tokens(history, tid * kTokens, a.history_len);
        const uint32_t length = a.history ? within(a.lengths, r, a.history_len, a.history_len) : 0u;
        const uint32_t prompt = within(a.prompt_lengths, r, 0u, length);
        uint32_t token = ~0u;   // of this thread's bias entry
        float bias = 0.0f;
        if (kLooked && tid < a.bias_len) {
            token = a.bias_ids[r * a.bias_ids_stride + tid] - lo;
            bias = a.bias[r * a.bias_stride + tid];
        }
        if (length > 0) {
            if (a.repetition) by = a.repetition[r];
            if (a.frequency) frequency = a.frequency[r];
            if (a.presence) presence = a.presence[r];
            inverse = fabsf(by) >= 0x1p-100f && fabsf(by) <= 0x1p100f ? 1.0f / by : __builtin_nanf("");
        }
        for (uint32_t i = tid; i < kVectors; i += kAdjustBlock) s_marks[i] = u32x4{0, 0, 0, 0};
        if constexpr (kLooked) {
            if (a.bias_len > 0) {
                for (uint32_t i = tid; i < kSlots; i += kAdjustBlock) {
                    s_token[i] = kFree;
                    s_entry[i] = 0;
                }
            }
        }
        __syncthreads();
        if constexpr (kLooked) {
            if (a.bias_len > 0) {
                uint32_t slot = token % kSlots;
                if (token < size) {
                    for (;; slot = (slot + 1) % kSlots) {   // there are more slots than entries
                        const uint32_t held = atomicCAS(&s_token[slot], kFree, token);
                        if (held == kFree || held == token) break;
                    }
                    atomicMax(&s_entry[slot], tid);   // the last entry counts
                    if constexpr (MARKS == kMarks16) atomicOr(&s_mark[token / 2], kBiased << token % 2 * 16);
                    else atomicOr(&s_mark[token], kBiased);
                }
                __syncthreads();
                if (token < size && s_entry[slot] == tid) s_bias[slot] = bias;
            }
        } else if (a.bias_ids) {
            for (uint32_t i = tid; i < a.bias_len; i += kAdjustBlock) {
                const uint32_t v = a.bias_ids[r * a.bias_ids_stride + i] - lo;
                if (v < size) atomicMax(&s_word[v], static_cast<Word>(i + 1));
            }
            __syncthreads();   // nothing is above the entries yet
        }
        for (uint32_t i0 = 0; i0 < length; i0 += kRound) {
            const Tokens now = next;
            const uint32_t i = i0 + tid * kTokens;
            if (i0 + kRound < length) next = load_tokens(history, i + kRound, a.history_len);
#pragma unroll
            for (int j = 0; j < kTokens; ++j) {
                const uint32_t v = now[j] - lo;   // a token that is none lies behind every slice
                if (v >= size || i + j >= length) continue;
                const bool before = i + j < prompt;
                if constexpr (MARKS == kMarks64) {
                    if (before) atomicOr(&s_word[v], kPrompt64);
                    else atomicAdd(&s_word[v], kOne);
                } else {
                    uint32_t* mark = &s_mark[MARKS == kMarks16 ? v / 2 : v];
                    const uint32_t shift = MARKS == kMarks16 ? v % 2 * 16 : 0;
                    if (before) atomicOr(mark, kPrompt << shift);
                    else atomicAdd(mark, 1u << shift);
                }
            }
        }
        __syncthreads();
    }

    // the bias of a token that has one
    auto bias_of = [&](uint32_t v) {
        uint32_t slot = v % kSlots;
        while (s_token[slot] != v) slot = (slot + 1) % kSlots;
        return s_bias[slot];
    };
#pragma unroll
    for (int h = 0; h < HOLD; ++h) {
        const uint32_t i = (h * kAdjustBlock + tid) * V;
        if (i >= size) break;
        float l[V];
        widen<T>(x[h], l);
        if constexpr (kLooked) {
            uint32_t m[V * kBits / 32], any = 0;
#pragma unroll
            for (uint32_t j = 0; j < V * kBits / 32; ++j) {
                m[j] = s_mark[i * kBits / 32 + j];
                any |= m[j];
            }
            if (any != 0) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const uint32_t w = MARKS == kMarks16 ? m[j / 2] >> (j % 2 * 16) & 0xFFFFu : m[j];
                    if (w == 0) continue;   // of all lanes: 256 rows of 131072, histories up to 500, 25.6 us for 27.8
                    l[j] = penalised(l[j], (w & ~kBiased) != 0, w & (kBiased - 1));
                    if (w & kBiased) l[j] += bias_of(i + j);
                }
            }
        }
        if constexpr (MARKS == kMarks64) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const Word w = s_word[i + j];
                if (w == 0) continue;
                const uint32_t entry = static_cast<uint32_t>(w & (kOne - 1));
                l[j] = penalised(l[j], w >= kOne, static_cast<uint32_t>((w & (kPrompt64 - 1)) >> 31));
                if (entry > 0) l[j] += a.bias[r * a.bias_stride + entry - 1];
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = (allowed[h] >> j) & 1u ? l[j] : -__builtin_huge_valf();
        store_some<V>(to + i, size - i, l);
    }
}

template <class T, class O, Marks MARKS, int HOLD>
void launch_as(const AdjustArgs& a, hipStream_t stream) {
    constexpr uint32_t kSlice = kAdjustBlock * HOLD * kVec<T>;
    const uint32_t slices = (a.vocab + kSlice - 1) / kSlice;
    adjust_kernel<T, O, MARKS, HOLD><<<many_blocks(static_cast<uint64_t>(a.rows) * slices), kAdjustBlock, 0, stream>>>(a, slices);
}

template <class T, class O>
hipError_t adjust_of(const AdjustArgs& a, hipStream_t stream) {
    const Marks marks = !a.history && !a.bias_ids ? kNoMarks : a.bias_len > kMaxLooked ? kMarks64
                        : a.history_len >= kMaxHistory16 ? kMarks32 : kMarks16;
    // two vectors a thread, where that leaves the chip 1024 blocks (four and eight leave a CU too few)
    const uint64_t vectors = static_cast<uint64_t>(a.rows) * ((a.vocab + kVec<T> - 1) / kVec<T>);
    const bool two = vectors >= uint64_t{2048} * kAdjustBlock;
    timing_before(stream, RS_KERNEL_ADJUST);
    switch (marks) {
        case kNoMarks: two ? launch_as<T, O, kNoMarks, 2>(a, stream) : launch_as<T, O, kNoMarks, 1>(a, stream); break;
        case kMarks16: two ? launch_as<T, O, kMarks16, 2>(a, stream) : launch_as<T, O, kMarks16, 1>(a, stream); break;
        case kMarks32: two ? launch_as<T, O, kMarks32, 2>(a, stream) : launch_as<T, O, kMarks32, 1>(a, stream); break;
        default: two ? launch_as<T, O, kMarks64, 2>(a, stream) : launch_as<T, O, kMarks64, 1>(a, stream); break;
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
