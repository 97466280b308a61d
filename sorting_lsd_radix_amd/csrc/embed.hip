// embed.hip -- rows of an embedding table by token, and the table's gradient.
//
// The gradient sorts the tokens with their positions (stably) and sums the
// rows of each token: a wave takes a piece of kPiece sorted positions and a
// chunk of 64 vectors of 16 bytes.  A token inside one piece is stored at once;
// of one that goes on, each piece keeps an f32 part, and the piece where the
// token begins joins them in order.  Nothing depends on the order in which
// blocks run.
#include "internal.hpp"
#include "rows_common.hpp"

namespace rs {

namespace {

constexpr int kEmbedBlock = 256;
constexpr int kEmbedWaves = kEmbedBlock / kWave;
constexpr uint32_t kPiece = 16;

template <class T>
constexpr int kVec = 16 / sizeof(T);

template <class T>
uint32_t chunks_of(uint32_t width) {
    return (width + kWave * kVec<T> - 1) / (kWave * kVec<T>);
}

template <class T, bool SCALED>
__global__ __launch_bounds__(kEmbedBlock) void embed_kernel(EmbedArgs a, uint32_t chunks) {
    constexpr int V = kVec<T>;
    const uint64_t unit = static_cast<uint64_t>(block_id()) * kEmbedWaves + threadIdx.x / kWave;
    const uint64_t i = unit / chunks;
    const uint32_t col = static_cast<uint32_t>(unit % chunks) * (kWave * V) + lane_id() * V;
    if (i >= a.n || col >= a.width) return;
    const uint32_t id = a.ids[i];
    const uint32_t left = a.width - col;
    const bool real = id < a.vocab;
    const T* from = static_cast<const T*>(a.table) + (real ? id : 0u) * a.table_stride + col;
    T* to = static_cast<T*>(a.out) + i * a.out_stride + col;
    if (SCALED) {
        float v[V] = {};
        if (real) {
            load_some<V>(from, left, 0.0f, v);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] *= a.scale;
        }
        store_some<V>(to, left, v);
    } else {
        copy_some<V>(from, real, to, left);
    }
}

// Sort keys: the tokens, `vocab` for those outside the table; values: positions.
__global__ __launch_bounds__(kEmbedBlock) void embed_keys_kernel(const uint32_t* __restrict__ ids, uint32_t n,
                                                                 uint32_t vocab, uint32_t* __restrict__ keys,
                                                                 uint32_t* __restrict__ at) {
    const uint64_t i = static_cast<uint64_t>(block_id()) * kEmbedBlock + threadIdx.x;
    if (i >= n) return;
    const uint32_t id = ids[i];
    keys[i] = id < vocab ? id : vocab;
    at[i] = static_cast<uint32_t>(i);
}

template <class T, class O>
__device__ __forceinline__ void store_row(const EmbedGradArgs& a, uint32_t id, uint32_t col, uint32_t left,
                                          float (&sum)[kVec<T>]) {
    constexpr int V = kVec<T>;
    O* to = static_cast<O*>(a.dtable) + id * a.dtable_stride + col;
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] *= a.scale;
    if (a.accumulate) {
        float old[V];
        load_some<V>(to, left, 0.0f, old);
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] += old[j];
    }
    store_some<V>(to, left, sum);
}

// Parts of tokens that cross pieces: two rows of `width` f32 for each piece,
// of its first token, if that began before, and of its last.
template <class T, class O>
__global__ __launch_bounds__(kEmbedBlock) void embed_sum_kernel(EmbedGradArgs a, uint32_t chunks,
                                                                const uint32_t* __restrict__ keys,
                                                                const uint32_t* __restrict__ at,
                                                                float* __restrict__ parts) {
    constexpr int V = kVec<T>;
    const uint64_t unit = static_cast<uint64_t>(block_id()) * kEmbedWaves + threadIdx.x / kWave;
    const uint64_t piece = unit / chunks;
    const uint64_t begin = piece * kPiece;
    if (begin >= a.n) return;
    const uint32_t end = a.n - begin < kPiece ? a.n : static_cast<uint32_t>(begin) + kPiece;
    const uint32_t col = static_cast<uint32_t>(unit % chunks) * (kWave * V) + lane_id() * V;
    const uint32_t left = col < a.width ? a.width - col : 0u;
    uint32_t id = keys[begin];
    bool before = begin > 0 && keys[begin - 1] == id;
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;
    for (uint32_t i = static_cast<uint32_t>(begin); i < end; ++i) {
        float v[V];
        load_some<V>(static_cast<const T*>(a.dout) + at[i] * a.dout_stride + col, left, 0.0f, v);
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] += v[j];
        const uint32_t next = i + 1 < a.n ? keys[i + 1] : ~0u;   // no key is ~0
        if (next == id && i + 1 < end) continue;
        const bool after = next == id;
        if (id < a.vocab) {
            if (!before && !after) store_row<T, O>(a, id, col, left, sum);
            else store_some<V>(parts + (2 * piece + (before ? 0 : 1)) * a.width + col, left, sum);
        }
        id = next;
        before = false;
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] = 0.0f;
    }
}

template <class T, class O>
__global__ __launch_bounds__(kEmbedBlock) void embed_join_kernel(EmbedGradArgs a, uint32_t chunks,
                                                                 const uint32_t* __restrict__ keys,
                                                                 const float* __restrict__ parts) {
    constexpr int V = kVec<T>;
    const uint64_t unit = static_cast<uint64_t>(block_id()) * kEmbedWaves + threadIdx.x / kWave;
    uint64_t piece = unit / chunks;
    const uint64_t begin = piece * kPiece;
    if (a.n <= kPiece || begin >= a.n - kPiece) return;   // the last piece's tokens end there
    const uint32_t id = keys[begin + kPiece - 1];
    if (id >= a.vocab || keys[begin + kPiece] != id) return;
    if (keys[begin] == id && begin > 0 && keys[begin - 1] == id) return;   // begins in an earlier piece
    const uint32_t col = static_cast<uint32_t>(unit % chunks) * (kWave * V) + lane_id() * V;
    const uint32_t left = col < a.width ? a.width - col : 0u;
    float sum[V];
    load_some<V>(parts + (2 * piece + 1) * a.width + col, left, 0.0f, sum);
    for (++piece; piece * kPiece < a.n && keys[piece * kPiece] == id; ++piece) {
        float v[V];
        load_some<V>(parts + 2 * piece * a.width + col, left, 0.0f, v);
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] += v[j];
    }
    store_row<T, O>(a, id, col, left, sum);
}

// Zeros in the rows of tokens that do not occur, a wave for each chunk of a row.
template <class O>
__global__ __launch_bounds__(kEmbedBlock) void embed_zero_kernel(EmbedGradArgs a, uint32_t chunks,
                                                                 const uint32_t* __restrict__ keys) {
    constexpr int V = kVec<O>;
    const uint64_t unit = static_cast<uint64_t>(block_id()) * kEmbedWaves + threadIdx.x / kWave;
    const uint64_t id = unit / chunks;
    if (id >= a.vocab) return;
    uint32_t lo = 0, hi = a.n;   // the first key that is not below id
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (keys[mid] < id) lo = mid + 1;
        else hi = mid;
    }
    if (lo < a.n && keys[lo] == id) return;
    const uint32_t col = static_cast<uint32_t>(unit % chunks) * (kWave * V) + lane_id() * V;
    if (col >= a.width) return;
    const float zero[V] = {};
    store_some<V>(static_cast<O*>(a.dtable) + id * a.dtable_stride + col, a.width - col, zero);
}

uint64_t pieces_of(uint64_t n) { return (n + kPiece - 1) / kPiece; }

size_t up256(size_t bytes) { return (bytes + 255) / 256 * 256; }

// Temp: keys, positions, both sorted, the sort's own temp, the parts.
struct Temp {
    size_t array, sort, parts;
    Temp(uint64_t n, uint32_t width) {
        array = up256(n * sizeof(uint32_t));
        sort = up256(sort_temp_bytes(n, true, SortKind{}));
        parts = n > kPiece ? up256(pieces_of(n) * 2 * width * sizeof(float)) : 0;
    }
    size_t bytes() const { return 4 * array + sort + parts; }
};

template <class T>
hipError_t embed_of(const EmbedArgs& a, hipStream_t stream) {
    const uint32_t chunks = chunks_of<T>(a.width);
    timing_before(stream, RS_KERNEL_EMBED);
    const auto kernel = a.scale == 1.0f ? embed_kernel<T, false> : embed_kernel<T, true>;
    kernel<<<many_blocks((static_cast<uint64_t>(a.n) * chunks + kEmbedWaves - 1) / kEmbedWaves), kEmbedBlock, 0,
             stream>>>(a, chunks);
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

template <class T, class O>
hipError_t embed_grad_of(const EmbedGradArgs& a, void* temp, hipStream_t stream) {
    const Temp size(a.n, a.width);
    char* base = static_cast<char*>(temp);
    uint32_t* keys_in = reinterpret_cast<uint32_t*>(base);
    uint32_t* at_in = reinterpret_cast<uint32_t*>(base + size.array);
    uint32_t* keys = reinterpret_cast<uint32_t*>(base + 2 * size.array);
    uint32_t* at = reinterpret_cast<uint32_t*>(base + 3 * size.array);
    void* sort_temp = base + 4 * size.array;
    float* parts = reinterpret_cast<float*>(base + 4 * size.array + size.sort);
    hipError_t e = hipSuccess;
    if (a.n > 0) {
        timing_before(stream, RS_KERNEL_EMBED_KEYS);
        embed_keys_kernel<<<many_blocks((a.n + uint64_t{kEmbedBlock} - 1) / kEmbedBlock), kEmbedBlock, 0, stream>>>(
            a.ids, a.n, a.vocab, keys_in, at_in);
        e = hipGetLastError();
        timing_after(stream);
        if (e != hipSuccess) return e;
        int bits = 1;
        while ((uint64_t{a.vocab} >> bits) != 0) ++bits;
        e = launch_sort(SortIo{keys_in, keys, nullptr, nullptr, at_in, at, a.n}, SortKind{}, 0, bits, sort_temp, stream);
        if (e != hipSuccess) return e;
    }
    const uint32_t chunks = chunks_of<T>(a.width);
    if (!a.accumulate) {
        const uint32_t out_chunks = chunks_of<O>(a.width);
        timing_before(stream, RS_KERNEL_EMBED_SUM);
        embed_zero_kernel<O><<<many_blocks((static_cast<uint64_t>(a.vocab) * out_chunks + kEmbedWaves - 1) / kEmbedWaves),
                               kEmbedBlock, 0, stream>>>(a, out_chunks, keys);
        e = hipGetLastError();
        timing_after(stream);
        if (e != hipSuccess) return e;
    }
    if (a.n == 0) return hipSuccess;
    const dim3 grid = many_blocks((pieces_of(a.n) * chunks + kEmbedWaves - 1) / kEmbedWaves);
    timing_before(stream, RS_KERNEL_EMBED_SUM);
    embed_sum_kernel<T, O><<<grid, kEmbedBlock, 0, stream>>>(a, chunks, keys, at, parts);
    e = hipGetLastError();
    timing_after(stream);
    if (e != hipSuccess || a.n <= kPiece) return e;
    timing_before(stream, RS_KERNEL_EMBED_JOIN);
    embed_join_kernel<T, O><<<grid, kEmbedBlock, 0, stream>>>(a, chunks, keys, parts);
    e = hipGetLastError();
    timing_after(stream);
    return e;
}

}  // namespace

hipError_t launch_embed(int elem_type, const EmbedArgs& a, hipStream_t stream) {
    if (a.n == 0) return hipSuccess;
    switch (elem_type) {
        case RS_ELEM_F32: return embed_of<float>(a, stream);
        case RS_ELEM_F16: return embed_of<_Float16>(a, stream);
        default: return embed_of<__bf16>(a, stream);
    }
}

size_t embed_grad_temp_bytes(uint64_t n, uint32_t vocab, uint32_t width) { return Temp(n, width).bytes(); }

hipError_t launch_embed_grad(int elem_type, int table_type, const EmbedGradArgs& a, void* temp, hipStream_t stream) {
    const bool f32 = table_type == RS_ELEM_F32;
    switch (elem_type) {
        case RS_ELEM_F32: return embed_grad_of<float, float>(a, temp, stream);
        case RS_ELEM_F16:
            return f32 ? embed_grad_of<_Float16, float>(a, temp, stream) : embed_grad_of<_Float16, _Float16>(a, temp, stream);
        default:
            return f32 ? embed_grad_of<__bf16, float>(a, temp, stream) : embed_grad_of<__bf16, __bf16>(a, temp, stream);
    }
}

}  // namespace rs
