// adjust.hip -- penalties of repeated tokens, biases and grammar masks on rows
// of logits, in one pass.
//
// A block takes a slice of a row's vocabulary.  It keeps a word for each token
// of the slice in LDS, marks there what the row's lists say of the slice's
// tokens (how often one occurs behind the prompt, whether in the prompt, the
// last bias entry that names it), with atomics whose order does not matter, and
// then passes once over its logits.
#include "internal.hpp"
#include "rows_common.hpp"

namespace rs {

namespace {

constexpr int kAdjustBlock = 256;

template <class T>
constexpr int kVec = 16 / sizeof(T);

// A token's word: from the low end a bias entry's index + 1, the occurrences
// behind the prompt, a bit for an occurrence in it.
template <class W>
struct Word;
template <>
struct Word<uint32_t> {
    static constexpr int kEntryBits = 16, kCountBits = 15;
};
template <>
struct Word<uint64_t> {
    static constexpr int kEntryBits = 31, kCountBits = 32;
};

// W = void: no lists.
template <class T, class O, class W>
__global__ __launch_bounds__(kAdjustBlock) void adjust_kernel(AdjustArgs a, uint32_t slices, uint32_t slice) {
    constexpr int V = kVec<T>;
    extern __shared__ uint64_t s_words[];
    W* word = reinterpret_cast<W*>(s_words);
    constexpr int kEntryBits = Word<W>::kEntryBits;
    constexpr W kOne = W{1} << kEntryBits;
    constexpr W kPrompt = kOne << Word<W>::kCountBits;
    const uint32_t b = block_id(), tid = threadIdx.x;
    const uint32_t r = b / slices;
    if (r >= a.rows) return;
    const uint32_t lo = b % slices * slice;
    const uint32_t size = a.vocab - lo < slice ? a.vocab - lo : slice;
    const bool lists = a.history || a.bias_ids;
    float by = 1.0f, frequency = 0.0f, presence = 0.0f;
    if (lists) {
        for (uint32_t i = tid; i < size; i += kAdjustBlock) word[i] = 0;
        __syncthreads();
        if (a.bias_ids) {
            for (uint32_t i = tid; i < a.bias_len; i += kAdjustBlock) {
                const uint32_t v = a.bias_ids[r * a.bias_ids_stride + i] - lo;
                if (v < size) atomicMax(&word[v], static_cast<W>(i + 1));
            }
            __syncthreads();
        }
        if (a.history) {
            auto within = [&](const int32_t* n, uint32_t all) {
                const int32_t x = n[r];
                return x < 0 ? 0u : static_cast<uint32_t>(x) < all ? static_cast<uint32_t>(x) : all;
            };
            const uint32_t length = a.lengths ? within(a.lengths, a.history_len) : a.history_len;
            const uint32_t prompt = a.prompt_lengths ? within(a.prompt_lengths, length) : 0u;
            for (uint32_t i = tid; i < length; i += kAdjustBlock) {
                const uint32_t v = a.history[r * a.history_stride + i] - lo;
                if (v >= size) continue;
                if (i < prompt) atomicOr(&word[v], kPrompt);
                else atomicAdd(&word[v], kOne);
            }
            if (a.repetition) by = a.repetition[r];
            if (a.frequency) frequency = a.frequency[r];
            if (a.presence) presence = a.presence[r];
            __syncthreads();
        }
    }
    const T* from = static_cast<const T*>(a.logits) + r * a.row_stride + lo;
    O* to = static_cast<O*>(a.out) + r * a.out_stride + lo;
    for (uint32_t i = tid * V; i < size; i += kAdjustBlock * V) {
        float x[V];
        load_some<V>(from + i, size - i, 0.0f, x);
        const uint32_t allowed = a.mask ? a.mask[r * a.mask_stride + (lo + i) / 32] >> ((lo + i) % 32) : ~0u;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const W w = lists && i + j < size ? word[i + j] : W{0};
            if (w != 0) {
                const uint32_t count = static_cast<uint32_t>((w & (kPrompt - 1)) >> kEntryBits);
                if (w >= kOne) x[j] = x[j] > 0.0f ? x[j] / by : x[j] * by;
                if (count > 0) x[j] -= fmaf(frequency, static_cast<float>(count), presence);
                const uint32_t entry = static_cast<uint32_t>(w & (kOne - 1));
                if (entry) x[j] += a.bias[r * a.bias_stride + entry - 1];
            }
            if (!((allowed >> j) & 1u)) x[j] = -__builtin_huge_valf();
        }
        store_some<V>(to + i, size - i, x);
    }
}

template <class T, class O>
hipError_t adjust_of(const AdjustArgs& a, hipStream_t stream) {
    // counts and entries of a wide word's fields only where the lists can be longer than a narrow one's
    const bool wide = a.history_len >= (1u << Word<uint32_t>::kCountBits) || a.bias_len >= (1u << Word<uint32_t>::kEntryBits);
    const bool lists = a.history || a.bias_ids;
    const uint32_t slice = wide ? 4096 : 8192;
    const uint32_t slices = (a.vocab + slice - 1) / slice;
    const size_t lds = lists ? slice * (wide ? 8 : 4) : 0;
    const dim3 grid = many_blocks(static_cast<uint64_t>(a.rows) * slices);
    timing_before(stream, RS_KERNEL_ADJUST);
    if (wide) adjust_kernel<T, O, uint64_t><<<grid, kAdjustBlock, lds, stream>>>(a, slices, slice);
    else adjust_kernel<T, O, uint32_t><<<grid, kAdjustBlock, lds, stream>>>(a, slices, slice);
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
