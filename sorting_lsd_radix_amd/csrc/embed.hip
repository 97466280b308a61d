// embed.hip -- rows of an embedding table by token, and the table's gradient.
//
// The gradient sorts the tokens with their positions (stably) and sums the
// rows of each token: a wave takes a piece of some sorted positions and a chunk
// of 64 vectors of 16 bytes.  A token inside one piece is stored at once; of one
// that goes on, each piece keeps an f32 part, and the block of the piece where the
// token begins joins them in order.  Nothing depends on the order in which
// blocks run.
//
// Rows without a token are zeros.  Where tokens are few for the table's rows, blocks
// beside the sort, whose launches are short chains of dependent steps, write all
// rows, which the sums then make good.  Otherwise the sort's first pass marks the
// tokens that occur, and the other rows are filled beside the sums (looking a row's
// mark up costs a tenth of the filling's rate).
//
// What bounds it: 131072 rows of 2048 bf16 and 16384 tokens take 125 us.  A trace, under
// which launches take some 4 % longer, has 101 for the sort's two launches with the filling (512 MB, 5.3
// TB/s), 23 for the sums, 7 for the join.  32003 rows of 1001 f32 and 50021 tokens take 85; the
// trace has 21 for the sort, 61 for the sums and zeros (318 MB, 5.2 TB/s), 8 for the join.  Rows by
// token: 32768 of 5120 f16 91 us (4.9 TB/s).
#include "internal.hpp"
#include "move_common.hpp"

namespace rs {

namespace {

hipError_t done(hipStream_t stream) {
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

// ---- rows by token ------------------------------------------------------------------

// A wave for each part of a row of more than 32 vectors.
template <class T, int U, bool SCALED>
__global__ __launch_bounds__(kMoveBlock) void embed_kernel(EmbedArgs a, uint32_t parts) {
    const uint32_t unit = block_id() * kMoveWaves + wave_id();
    const uint32_t i = unit / parts;
    if (i >= a.n) return;
    const uint32_t id = a.ids[i];
    const RowPart<T, U> row(unit % parts, a.width);
    typename RowPart<T, U>::Vec r[U] = {};
    if (id < a.vocab) {
        row.load(static_cast<const T*>(a.table) + id * a.table_stride, r);
        if (SCALED) {
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = scaled<T>(r[u], a.scale);
        }
    }
    row.store(static_cast<T*>(a.out) + i * a.out_stride, r);
}

// L lanes a row, up to L vectors.
template <class T, int L, bool SCALED>
__global__ __launch_bounds__(kMoveBlock) void embed_narrow_kernel(EmbedArgs a) {
    constexpr int V = kVec<T>;
    const uint64_t i = static_cast<uint64_t>(block_id()) * (kMoveBlock / L) + threadIdx.x / L;
    const uint32_t col = threadIdx.x % L * V;
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

template <class T, bool SCALED>
hipError_t embed_of(const EmbedArgs& a, hipStream_t stream) {
    const uint32_t vectors = static_cast<uint32_t>(up(a.width, kVec<T>));
    timing_before(stream, RS_KERNEL_EMBED);
    if (vectors <= 32) {   // 32768 rows of 32: 6.9 us, a wave each 7.9
        const uint32_t lanes = vectors <= 4 ? 4 : vectors <= 16 ? 16 : 32;
        const auto kernel = lanes == 4 ? embed_narrow_kernel<T, 4, SCALED> : lanes == 16 ? embed_narrow_kernel<T, 16, SCALED>
                                                                                         : embed_narrow_kernel<T, 32, SCALED>;
        kernel<<<many_blocks(up(a.n, kMoveBlock / lanes)), kMoveBlock, 0, stream>>>(a);
    } else {
        const Split s = split_rows(vectors, a.n, 2);
        const auto kernel = s.unroll == 1 ? embed_kernel<T, 1, SCALED> : embed_kernel<T, 2, SCALED>;
        kernel<<<many_blocks(up(static_cast<uint64_t>(a.n) * s.parts, kMoveWaves)), kMoveBlock, 0, stream>>>(a, s.parts);
    }
    return done(stream);
}

// ---- zeros in rows without a token ------------------------------------------------------

// Rows first .. last of a table, `each` (at most 64) a wave, on 2^lanes_log2
// lanes a row; those of tokens that occur are left out, where that is known.
struct Zeros {
    void* table;
    uint64_t stride;
    const uint8_t* occurs;
    uint32_t first, last, width, each, lanes_log2;
};

// All rows first .. last of a table without gaps, a store for each lane: plain fills of
// 1 GB reach 6.9 TB/s so and 6.0 with four stores a lane; beside the sort of 1000
// tokens 512 MB take 103 us for 108.
template <class O>
__device__ __forceinline__ void zero_flat(const Zeros& z, uint64_t wave) {
    constexpr int V = kVec<O>;
    const uint64_t at = static_cast<uint64_t>(z.first) * z.width + (wave * kWave + lane_id()) * V;
    const uint64_t end = static_cast<uint64_t>(z.last) * z.width;
    const float zero[V] = {};
    if (at < end) store_some<V>(static_cast<O*>(z.table) + at, end - at < V ? static_cast<uint32_t>(end - at) : V, zero);
}

template <class O>
__device__ __forceinline__ void zero_rows(const Zeros& z, uint64_t wave) {
    constexpr int V = kVec<O>;
    const uint32_t lane = lane_id();
    if (z.occurs == nullptr && z.stride == z.width) return zero_flat<O>(z, wave);
    const uint64_t row0 = z.first + wave * z.each;
    if (row0 >= z.last) return;
    const uint32_t n = z.last - row0 < z.each ? z.last - static_cast<uint32_t>(row0) : z.each;
    const uint64_t rows = ballot(lane < n && !(z.occurs && z.occurs[row0 + lane]));
    const uint32_t groups = kWave >> z.lanes_log2;
    const float zero[V] = {};
    for (uint32_t s = 0; s < n; s += groups) {
        const uint32_t r = s + (lane >> z.lanes_log2);
        if (r >= n || !((rows >> r) & 1u)) continue;
        O* to = static_cast<O*>(z.table) + (row0 + r) * z.stride;
        for (uint64_t c = (lane & ((1u << z.lanes_log2) - 1)) * V; c < z.width; c += static_cast<uint64_t>(V) << z.lanes_log2)
            store_some<V>(to + c, z.width - static_cast<uint32_t>(c), zero);
    }
}

// Waves for rows first .. last.
template <class O>
uint64_t zero_waves(const Zeros& z) {
    const uint64_t rows = z.last - z.first;
    return z.occurs == nullptr && z.stride == z.width ? up(rows * z.width, kWave * kVec<O>) : up(rows, z.each);
}
// Rows whose zeros are at most `waves` waves' work.  A grid's 2^26 waves have 2^32
// lanes and a row at most 2^28 vectors, so there are some.
template <class O>
uint64_t zero_rows_of(const Zeros& z, uint64_t waves) {
    return z.occurs == nullptr && z.stride == z.width ? waves * (kWave * kVec<O>) / z.width : waves * z.each;
}

// ---- the sort -----------------------------------------------------------------------------
//
// A stable counting sort by digits of up to 10 bits, lowest first.  A block
// ranks a tile of keys as group.hip does: wave w holds the w-th run of 64 ITEMS
// keys, 64 a row, which it ranks row by row.

constexpr int kSortBlock = 1024;
constexpr int kSortWaves = kSortBlock / kWave;
constexpr uint32_t kMaxBits = 10;
constexpr uint32_t kMaxTiles = 128;   // each block sums the counts of all tiles
constexpr uint32_t kMaxSortGrid = (1u << 22) - 1;   // blocks: a grid dimension holds less than 2^32 work items

struct Pass {
    const uint32_t* keys;   // the tokens in the first pass
    const uint32_t* at;     // their positions, null in the first pass
    uint32_t* keys_out;
    uint32_t* at_out;
    uint32_t* counts;       // [tiles][bins], or null: each tile counts the keys itself
    uint8_t* occurs;        // [vocab]: a byte for each token that occurs
    uint32_t n, vocab, tiles, shift, bits;
    bool clear, mark;       // whether this launch clears those bytes, and sets them
};

// Clears the bytes of the tokens, beside the tiles' other work.
__device__ __forceinline__ void clear_occurs(const Pass& p) {
    const uint32_t words = static_cast<uint32_t>((static_cast<uint64_t>(p.vocab) + 3) / 4);
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kSortBlock + threadIdx.x; i < words; i += static_cast<uint64_t>(gridDim.x) * kSortBlock)
        reinterpret_cast<uint32_t*>(p.occurs)[i] = 0;
}

// A key: the token, `vocab` for one outside the table.
__device__ __forceinline__ uint32_t key_of(const Pass& p, uint64_t i) {
    const uint32_t k = p.keys[i];
    return k < p.vocab ? k : p.vocab;
}

template <class O, int ITEMS>
__global__ __launch_bounds__(kSortBlock) void embed_count_kernel(Pass p, Zeros z) {
    __shared__ uint32_t s_count[1u << kMaxBits];
    const uint32_t tid = threadIdx.x;
    if (p.clear) clear_occurs(p);
    if (blockIdx.x >= p.tiles) return zero_rows<O>(z, static_cast<uint64_t>(blockIdx.x - p.tiles) * kSortWaves + wave_id());
    const uint32_t base = blockIdx.x * (kSortBlock * ITEMS);
    s_count[tid] = 0;
    uint32_t d[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const uint32_t i = base + j * kSortBlock + tid;
        d[j] = i < p.n ? (key_of(p, i) >> p.shift) & ((1u << p.bits) - 1) : ~0u;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j)
        if (d[j] != ~0u) atomicAdd(&s_count[d[j]], 1u);
    __syncthreads();
    if (tid < (1u << p.bits)) p.counts[(blockIdx.x << p.bits) + tid] = s_count[tid];
}

template <class O, int ITEMS>
__global__ __launch_bounds__(kSortBlock) void embed_place_kernel(Pass p, Zeros z) {
    __shared__ uint16_t s_count[kSortWaves][1u << kMaxBits];
    __shared__ uint32_t s_part[2][kSortBlock];
    __shared__ uint32_t s_base[1u << kMaxBits];
    __shared__ uint32_t s_wave[kSortWaves];
    const uint32_t tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    const uint32_t tile = blockIdx.x;
    if (tile >= p.tiles) return zero_rows<O>(z, static_cast<uint64_t>(tile - p.tiles) * kSortWaves + wave_id());
    if (p.clear) clear_occurs(p);
    const uint32_t bins = 1u << p.bits;
    const uint32_t base = tile * (kSortBlock * ITEMS) + wave * (kWave * ITEMS) + lane;
    uint32_t key[ITEMS], at[ITEMS], rank[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const uint32_t i = base + j * kWave;
        key[j] = i < p.n ? key_of(p, i) : ~0u;
        at[j] = i < p.n && p.at ? p.at[i] : i;
    }
    for (uint32_t x = lane; x < bins; x += kWave) s_count[wave][x] = 0;
    if (p.tiles > 1 && p.counts == nullptr) {
        // all keys, and those of earlier tiles; the digit of a wave's first lane, which may be
        // every lane's, is counted once for all of them
        s_part[0][tid] = s_part[1][tid] = 0;
        __syncthreads();
        const uint32_t here = tile * (kSortBlock * ITEMS);
        for (uint32_t i0 = 0; i0 < p.n; i0 += kSortBlock * 4) {
            uint32_t d[4];
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                const uint32_t i = i0 + j * kSortBlock + tid;
                d[j] = i < p.n ? (key_of(p, i) >> p.shift) & (bins - 1) : ~0u;
            }
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                const bool earlier = i0 + j * kSortBlock + tid < here;   // of a whole wave or none
                const bool with_first = d[j] == __builtin_amdgcn_readfirstlane(d[j]);
                const uint64_t same = ballot(with_first);
                const uint32_t n = with_first ? __builtin_popcountll(same) : 1;
                if (d[j] != ~0u && (!with_first || lane == 0)) {
                    atomicAdd(&s_part[1][d[j]], n);
                    if (earlier) atomicAdd(&s_part[0][d[j]], n);
                }
            }
        }
    } else if (p.tiles > 1) {
        // counts of the tiles: thread (slice q, bin) sums every slices-th tile
        const uint32_t slices = kSortBlock >> p.bits;
        const uint32_t bin = tid & (bins - 1), q = tid >> p.bits;
        constexpr uint32_t kAhead = 8;   // loads in flight: of the last tile again behind the end
        uint32_t before = 0, all = 0;
        for (uint32_t t0 = q; t0 < p.tiles; t0 += kAhead * slices) {
            uint32_t n[kAhead];
#pragma unroll
            for (uint32_t j = 0; j < kAhead; ++j) {
                const uint32_t t = t0 + j * slices;
                n[j] = p.counts[((t < p.tiles ? t : p.tiles - 1) << p.bits) + bin];
            }
#pragma unroll
            for (uint32_t j = 0; j < kAhead; ++j) {
                const uint32_t t = t0 + j * slices;
                all += t < p.tiles ? n[j] : 0u;
                before += t < tile ? n[j] : 0u;
            }
        }
        s_part[0][tid] = before;
        s_part[1][tid] = all;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const bool real = key[j] != ~0u;
        const uint32_t d = (key[j] >> p.shift) & (bins - 1);
        rank[j] = rank_among(s_count[wave], real, d, p.bits);
    }
    __syncthreads();
    uint32_t before = 0, total = 0;
    if (tid < bins) {
#pragma unroll
        for (uint32_t w = 0; w < kSortWaves; ++w) {
            const uint32_t n = s_count[w][tid];
            s_count[w][tid] = static_cast<uint16_t>(total);
            total += n;
        }
        if (p.tiles > 1) {
            total = 0;
            for (uint32_t x = tid; x < (p.counts ? kSortBlock : bins); x += bins) {
                before += s_part[0][x];
                total += s_part[1][x];
            }
        }
    }
    const uint32_t incl = wave_inclusive_sum(total);
    if (lane == kWave - 1) s_wave[wave] = incl;
    __syncthreads();
    uint32_t start = incl - total;
    for (uint32_t w = 0; w < wave; ++w) start += s_wave[w];
    if (tid < bins) s_base[tid] = start + before;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        if (key[j] == ~0u) continue;
        const uint32_t d = (key[j] >> p.shift) & (bins - 1);
        const uint32_t to = s_base[d] + s_count[wave][d] + rank[j];
        p.keys_out[to] = key[j];
        p.at_out[to] = at[j];
        if (p.mark && key[j] < p.vocab) p.occurs[key[j]] = 1;   // from all that do, the same byte
    }
}

// Sort keys and positions for the library's sort, which takes over above
// kMaxTiles tiles of 4096 tokens.
__global__ __launch_bounds__(kSortBlock) void embed_keys_kernel(Pass p) {
    const uint64_t i = static_cast<uint64_t>(block_id()) * kSortBlock + threadIdx.x;
    if (p.clear) {
        const uint64_t step = static_cast<uint64_t>(gridDim.x) * gridDim.y * kSortBlock;
        const uint64_t words = (static_cast<uint64_t>(p.vocab) + 3) / 4;
        for (uint64_t w = i; w < words; w += step) reinterpret_cast<uint32_t*>(p.occurs)[w] = 0;
    }
    if (i >= p.n) return;
    p.keys_out[i] = key_of(p, i);
    p.at_out[i] = static_cast<uint32_t>(i);
}

__global__ __launch_bounds__(kSortBlock) void embed_mark_kernel(Pass p) {
    const uint64_t i = static_cast<uint64_t>(block_id()) * kSortBlock + threadIdx.x;
    if (i < p.n && p.keys[i] < p.vocab) p.occurs[p.keys[i]] = 1;
}

// ---- the sums -------------------------------------------------------------------------------

// A lane's vector of the rows.  With WIDE the rows have a whole one, and the last
// begins where a whole one is left (as in RowPart): what it holds of the vector
// before is summed twice, to the same value.
template <class T, bool WIDE>
struct Columns {
    static constexpr int V = kVec<T>;
    using Vec = AnyVec<16>::V;
    uint32_t at, left, twice;   // first element, elements that the row has from there, those of the vector before

    __device__ __forceinline__ Columns(uint32_t vector, uint32_t width) {
        const uint32_t c = vector * V;
        at = WIDE && c > width - V ? width - V : c;
        left = c < width ? width - at : 0u;
        twice = c - at;
    }
    __device__ __forceinline__ Vec load(const T* row) const {
        if (WIDE) return __builtin_nontemporal_load(reinterpret_cast<const Vec*>(row + at));
        float x[V];
        load_some<V>(row + at, left, 0.0f, x);
        return narrow<T>(x);   // exact: they are T's
    }
    template <class P>
    __device__ __forceinline__ void store(P* row, const float (&x)[V]) const {
        if (left) store_some<V>(row + at, WIDE ? V : left, x);
    }
};

template <class T, class O, bool WIDE>
__device__ __forceinline__ void store_row(const EmbedGradArgs& a, uint32_t id, const Columns<T, WIDE>& c, float (&sum)[kVec<T>]) {
    constexpr int V = kVec<T>;
    O* row = static_cast<O*>(a.dtable) + id * a.dtable_stride;
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] *= a.scale;
    if (!a.accumulate) return c.store(row, sum);
    // each element by one lane alone
#pragma unroll
    for (uint32_t j = 0; j < V; ++j)
        if (j >= c.twice && j < c.left) row[c.at + j] = static_cast<O>(static_cast<float>(row[c.at + j]) + sum[j]);
}

struct Sorted {
    const uint32_t* keys;
    const uint32_t* at;
    float* parts;      // [pieces][2][width]: of a piece's first token, if it began before, and of its last
    uint32_t piece;    // positions of a piece, at most 64
    uint32_t chunks;   // of a row, or 1 where L lanes have it all
};

constexpr int kInFlight = 8;   // rows; 4 and 16 are within 2 %

// L lanes take a piece and 64 vectors of the rows, or, L < 64, all of them.
// Blocks behind the last piece fill the rows without tokens.
template <class T, class O, int L>
__global__ __launch_bounds__(kMoveBlock) void embed_sum_kernel(EmbedGradArgs a, Sorted s, Zeros z, uint32_t sums, uint32_t fill) {
    constexpr int V = kVec<T>;
    using Cols = Columns<T, L == kWave>;
    if (block_id() >= sums) {
        if (block_id() - sums < fill) zero_rows<O>(z, static_cast<uint64_t>(block_id() - sums) * kMoveWaves + wave_id());
        return;
    }
    const uint32_t unit = block_id() * (kMoveBlock / L) + (L == kWave ? wave_id() : threadIdx.x / L);
    const uint32_t piece = unit / s.chunks;
    const uint64_t begin = static_cast<uint64_t>(piece) * s.piece;
    if (begin >= a.n) return;
    uint32_t count = a.n - begin < s.piece ? a.n - static_cast<uint32_t>(begin) : s.piece;
    const uint32_t lane = threadIdx.x % L;
    const Cols cols(unit % s.chunks * L + lane, a.width);
    const T* rows = static_cast<const T*>(a.dout);
    const uint32_t* keys = s.keys + begin;
    const uint32_t* ats = s.at + begin;
    const uint32_t next = begin + count < a.n ? keys[count] : ~0u;   // no key is ~0
    bool before = begin > 0 && s.keys[begin - 1] == keys[0];
    // with a wave a piece, its keys and positions are in the lanes
    uint32_t lane_key = ~0u, lane_at = 0;
    if (L == kWave) {
        if (lane < count) {
            lane_key = keys[lane];
            lane_at = ats[lane];
        }
        count = __builtin_popcountll(ballot(lane_key < a.vocab));   // the others are last
        arrived(lane_key, lane_at);
    }
    auto key = [&](uint32_t i) { return L == kWave ? lane_value(lane_key, i) : keys[i]; };
    auto at = [&](uint32_t i) { return L == kWave ? lane_value(lane_at, i) : ats[i]; };
    float sum[V] = {};
    for (uint32_t i0 = 0; i0 < count; i0 += kInFlight) {
        typename Cols::Vec r[kInFlight];
#pragma unroll
        for (uint32_t b = 0; b < kInFlight; ++b)   // the last row again behind the end: no branch between the loads
            r[b] = cols.load(rows + at(i0 + b < count ? i0 + b : count - 1) * a.dout_stride);
#pragma unroll
        for (uint32_t b = 0; b < kInFlight; ++b) {
            const uint32_t i = i0 + b;
            if (i >= count) break;
            const uint32_t id = key(i);
            if (L < kWave && id >= a.vocab) break;
            float x[V];
            widen<T>(r[b], x);
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] += x[j];
            const bool last = i + 1 == s.piece || begin + i + 1 == a.n;
            const uint32_t then = last ? next : i + 1 < count ? key(i + 1) : ~0u;
            if (then == id && !last) continue;
            if (!before && then != id) store_row<T, O>(a, id, cols, sum);
            else cols.store(s.parts + (static_cast<uint64_t>(piece) * 2 + (before ? 0 : 1)) * a.width, sum);
            before = false;
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] = 0.0f;
        }
    }
}

constexpr int kJoinBlock = 1024;
constexpr uint32_t kFewParts = 8;   // that L lanes join by themselves

// The sum of parts first .. stop of a token that begins in `piece`: its last
// token's, then the first ones' of the pieces behind.
template <class Cols>
__device__ __forceinline__ void sum_parts(const Sorted& s, uint32_t width, uint32_t piece, uint32_t first, uint32_t stop,
                                          const Cols& cols, float (&sum)[Cols::V]) {
    constexpr int V = Cols::V;
    constexpr uint32_t kAhead = 4;
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;
    for (uint32_t i0 = first; i0 < stop; i0 += kAhead) {
        float r[kAhead][V];
#pragma unroll
        for (uint32_t b = 0; b < kAhead; ++b)
            if (i0 + b < stop)
                load_some<V>(s.parts + (static_cast<uint64_t>(piece + i0 + b) * 2 + (i0 + b == 0 ? 1 : 0)) * width + cols.at,
                             cols.left, 0.0f, r[b]);
#pragma unroll
        for (uint32_t b = 0; b < kAhead; ++b) {
            if (i0 + b >= stop) break;
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] += r[b][j];
        }
    }
}

// L lanes for each piece (and 64 vectors): if a token begins in it and goes on,
// they join its parts, or, if there are many, all of the block do, a run of
// them each, then the runs.
template <class T, class O, int L>
__global__ __launch_bounds__(kJoinBlock) void embed_join_kernel(EmbedGradArgs a, Sorted s) {
    constexpr int V = kVec<T>;
    constexpr uint32_t kWorkers = kJoinBlock / L;
    __shared__ float s_sum[kWorkers][L * V];
    __shared__ uint32_t s_many, s_piece[kWorkers], s_count[kWorkers], s_id[kWorkers];   // tokens of many parts
    const uint32_t worker = threadIdx.x / L, lane = threadIdx.x % L;
    const uint32_t piece0 = block_id() / s.chunks * kWorkers;
    const Columns<T, L == kWave> cols(block_id() % s.chunks * L + lane, a.width);
    const uint32_t piece = piece0 + worker;
    const uint64_t end = (static_cast<uint64_t>(piece) + 1) * s.piece;
    uint32_t count = 0, id = a.vocab;
    if (threadIdx.x == 0) s_many = 0;
    __syncthreads();
    if (end < a.n) {   // the last piece's tokens end there
        const uint64_t begin = end - s.piece;
        id = s.keys[end - 1];
        const bool goes_on = s.keys[end] == id;
        const bool whole = s.keys[begin] == id;
        if (id < a.vocab && goes_on && !(whole && begin > 0 && s.keys[begin - 1] == id)) {
            // pieces that begin with the token: behind `piece` up to the last one, found by halving
            uint32_t lo = piece + 1, hi = static_cast<uint32_t>((a.n - 1) / s.piece);
            if (hi - lo > kFewParts && s.keys[static_cast<uint64_t>(lo + kFewParts) * s.piece] != id) hi = lo + kFewParts - 1;
            while (lo < hi) {
                const uint32_t mid = hi - (hi - lo) / 2;
                if (s.keys[static_cast<uint64_t>(mid) * s.piece] == id) lo = mid;
                else hi = mid - 1;
            }
            count = lo - piece + 1;
        }
    }
    float sum[V];
    if (count > 0 && count <= kFewParts) {
        sum_parts(s, a.width, piece, 0, count, cols, sum);
        store_row<T, O>(a, id, cols, sum);
    }
    if (lane == 0 && count > kFewParts) {   // in any order: each token has its own row
        const uint32_t i = atomicAdd(&s_many, 1u);
        s_piece[i] = piece;
        s_count[i] = count;
        s_id[i] = id;
    }
    __syncthreads();
    const uint32_t many = s_many;
    for (uint32_t i = 0; i < many; ++i) {
        count = s_count[i];
        const uint32_t run = (count + kWorkers - 1) / kWorkers;
        const uint32_t workers = (count + run - 1) / run;
        if (worker < workers) {
            sum_parts(s, a.width, s_piece[i], worker * run, worker + 1 < workers ? (worker + 1) * run : count, cols, sum);
#pragma unroll
            for (int j = 0; j < V; ++j) s_sum[worker][j * L + lane] = sum[j];
        }
        __syncthreads();
        if (worker == 0) {
            for (uint32_t x = 1; x < workers; ++x) {
#pragma unroll
                for (int j = 0; j < V; ++j) sum[j] += s_sum[x][j * L + lane];
            }
            store_row<T, O>(a, s_id[i], cols, sum);
        }
        __syncthreads();
    }
}

// ---- launches ---------------------------------------------------------------------------------

uint32_t sort_items(uint64_t n) { return n <= kMaxTiles * kSortBlock ? 1 : 4; }
bool own_sort(uint64_t n) { return n <= uint64_t{kMaxTiles} * kSortBlock * 4; }
// Whether all rows are filled beside the sort, or beside the sums those that have no
// token.  With a quarter as many tokens as rows, 131072 rows of 2048 bf16 take 149 us and 159, 32000
// of 1001 f32 42.3 and 48.5, 8000 of 8192 bf16 40.8 and 43.3, 50000 of 512 f32 44.4 and 44.4,
// 262144 of 64 f16 51.4 and 51.3; with half as many 186 and 192, 58.8 and 57.8, 53.6 and 54.9,
// 52.5 and 51.0, 66.6 and 67.8: by then either may be ahead.
bool few_tokens(uint64_t n, uint32_t vocab) { return own_sort(n) && n > 0 && n <= vocab / 4; }
// Lanes that take a row's vectors of T, 64 for one of several chunks, and the chunks.
struct Lanes {
    uint32_t lanes, chunks;
};
Lanes lanes_of(uint64_t vectors) {
    if (vectors <= 4) return {4, 1};
    if (vectors <= 16) return {16, 1};
    return {kWave, static_cast<uint32_t>(up(vectors, kWave))};
}

// Positions of a piece: 8 to 64, so that 4096 waves or more fill the chip (with 2048
// 16384 tokens of 2048 bf16 take 148 us for 142, with 8192 150; 100000 of 16 f32 64 for 46).
uint32_t piece_of(uint64_t n, uint64_t vectors) {
    const Lanes l = lanes_of(vectors);
    uint32_t piece = 8;
    while (piece < 64 && n * l.chunks * l.lanes / kWave >= uint64_t{piece} * 2 * 4096) piece *= 2;
    return piece;
}

size_t up256(size_t bytes) { return (bytes + 255) / 256 * 256; }

// Temp: keys and positions twice, the tiles' counts or the library sort's own
// temp, which tokens occur, the parts.
struct Temp {
    size_t array, sort, occurs, parts;
    uint32_t piece;
    Temp(uint64_t n, uint32_t vocab, uint32_t width, uint32_t vector) {
        array = up256(n * sizeof(uint32_t));
        sort = own_sort(n) ? kMaxTiles * sizeof(uint32_t) << kMaxBits : up256(sort_temp_bytes(n, true, SortKind{}));
        occurs = up256(vocab);
        piece = piece_of(n, up(width, vector));
        parts = n > piece ? up256(up(n, piece) * 2 * width * sizeof(float)) : 0;
    }
    size_t bytes() const { return 4 * array + sort + occurs + parts; }
};

template <class O>
hipError_t sort_tokens(const EmbedGradArgs& a, Pass p, uint32_t* const (&keys)[2], uint32_t* const (&at)[2], Zeros& z,
                       bool fill, int* last, hipStream_t stream) {
    uint32_t bits = 1;
    while ((uint64_t{a.vocab} >> bits) != 0) ++bits;
    const uint32_t passes = (bits + kMaxBits - 1) / kMaxBits;
    const uint32_t each_bits = (bits + passes - 1) / passes;
    const uint32_t items = sort_items(a.n);
    p.tiles = static_cast<uint32_t>(up(a.n, uint64_t{kSortBlock} * items));
    const bool marks = p.clear;
    // With a launch for the tiles' counts, or, of few tiles, each counts all keys itself: 3 tiles 25.7 us
    // for 28.2 in all, 10 tiles 34.5 for 32.4; beside the filling, which hides it, 16 tiles 125.7 for
    // 127.5.  Where one pass has to clear the marks before several tiles set them, the launch is needed.
    const bool counts = p.tiles > (fill ? 16u : 4u) || (p.tiles > 1 && passes == 1 && marks);
    uint32_t* const tile_counts = p.counts;
    uint32_t launches = passes * (counts ? 2 : 1);
    // the next rows to be filled beside a launch, no more than its grid holds: their
    // blocks, and their end in z
    auto beside = [&] {
        z.first = z.last;
        const uint64_t left = fill ? a.vocab - z.first : 0, share = launches > 1 ? up(left, launches) : left;
        const uint64_t most = zero_rows_of<O>(z, uint64_t{kMaxSortGrid - kMaxTiles} * kSortWaves);
        if (launches > 1) --launches;
        z.last += static_cast<uint32_t>(share < most ? share : most);
        return static_cast<uint32_t>(up(zero_waves<O>(z), kSortWaves));
    };
    for (uint32_t k = 0; k < passes; ++k) {
        p.shift = k * each_bits;
        p.bits = bits - p.shift < each_bits ? bits - p.shift : each_bits;
        p.keys = k == 0 ? a.ids : keys[(k - 1) & 1];
        p.at = k == 0 ? nullptr : at[(k - 1) & 1];
        p.keys_out = keys[k & 1];
        p.at_out = at[k & 1];
        p.counts = counts ? tile_counts : nullptr;
        p.clear = marks && k == 0;
        p.mark = false;
        if (counts) {
            const uint32_t more = beside();
            timing_before(stream, RS_KERNEL_EMBED_SORT);
            const auto kernel = items == 1 ? embed_count_kernel<O, 1> : embed_count_kernel<O, 4>;
            kernel<<<dim3(p.tiles + more), kSortBlock, 0, stream>>>(p, z);
            const hipError_t e = done(stream);
            if (e != hipSuccess) return e;
        }
        if (counts) p.clear = false;
        p.mark = marks && k == (counts ? 0 : passes - 1);
        const uint32_t more = beside();
        timing_before(stream, RS_KERNEL_EMBED_SORT);
        const auto kernel = items == 1 ? embed_place_kernel<O, 1> : embed_place_kernel<O, 4>;
        kernel<<<dim3(p.tiles + more), kSortBlock, 0, stream>>>(p, z);
        const hipError_t e = done(stream);
        if (e != hipSuccess) return e;
        *last = k & 1;
    }
    // of a table past 64 GB a launch, the rest: by itself, since the sums write rows
    p.tiles = 0;
    while (fill && z.last < a.vocab) {
        const uint32_t more = beside();
        timing_before(stream, RS_KERNEL_EMBED_SORT);
        embed_count_kernel<O, 1><<<dim3(more), kSortBlock, 0, stream>>>(p, z);
        const hipError_t e = done(stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t sort_many_tokens(const EmbedGradArgs& a, Pass p, uint32_t* const (&keys)[2], uint32_t* const (&at)[2], void* temp,
                            hipStream_t stream) {
    p.keys = a.ids;
    p.keys_out = keys[0];
    p.at_out = at[0];
    const dim3 grid = many_blocks(up(a.n, kSortBlock));
    timing_before(stream, RS_KERNEL_EMBED_SORT);
    embed_keys_kernel<<<grid, kSortBlock, 0, stream>>>(p);
    hipError_t e = done(stream);
    if (e != hipSuccess) return e;
    if (p.clear) {
        p.keys = keys[0];
        timing_before(stream, RS_KERNEL_EMBED_SORT);
        embed_mark_kernel<<<grid, kSortBlock, 0, stream>>>(p);
        e = done(stream);
        if (e != hipSuccess) return e;
    }
    int bits = 1;
    while ((uint64_t{a.vocab} >> bits) != 0) ++bits;
    return launch_sort(SortIo{keys[0], keys[1], nullptr, nullptr, at[0], at[1], a.n}, SortKind{}, 0, bits, temp, stream);
}

template <class T, class O, int L>
hipError_t sum_tokens(const EmbedGradArgs& a, Sorted s, const Zeros& z, hipStream_t stream) {
    const uint64_t pieces = up(a.n, s.piece);
    const uint32_t sums = static_cast<uint32_t>(up(pieces * s.chunks, kMoveBlock / L));
    const uint32_t fill = static_cast<uint32_t>(up(zero_waves<O>(z), kMoveWaves));
    hipError_t e = hipSuccess;
    if (sums + fill > 0) {
        timing_before(stream, RS_KERNEL_EMBED_SUM);
        embed_sum_kernel<T, O, L><<<many_blocks(uint64_t{sums} + fill), kMoveBlock, 0, stream>>>(a, s, z, sums, fill);
        e = done(stream);
    }
    if (e != hipSuccess || pieces <= 1) return e;
    timing_before(stream, RS_KERNEL_EMBED_JOIN);
    embed_join_kernel<T, O, L><<<many_blocks(up(pieces, kJoinBlock / L) * s.chunks), kJoinBlock, 0, stream>>>(a, s);
    return done(stream);
}

template <class T, class O>
hipError_t embed_grad_of(const EmbedGradArgs& a, void* temp, hipStream_t stream) {
    const Temp size(a.n, a.vocab, a.width, kVec<T>);
    char* base = static_cast<char*>(temp);
    auto words = [&](size_t offset) { return reinterpret_cast<uint32_t*>(base + offset); };
    uint32_t* const keys[2] = {words(0), words(2 * size.array)};
    uint32_t* const at[2] = {words(size.array), words(3 * size.array)};
    void* sort = base + 4 * size.array;
    uint8_t* occurs = reinterpret_cast<uint8_t*>(base + 4 * size.array + size.sort);
    Sorted s{keys[0], at[0], reinterpret_cast<float*>(occurs + size.occurs), size.piece, 1};

    Zeros z{a.dtable, a.dtable_stride, nullptr, 0, 0, a.width, 1, 6};
    const uint64_t row_bytes = uint64_t{a.width} * sizeof(O);
    while (z.each < 64 && z.each * row_bytes < 4096) z.each *= 2;
    while (z.lanes_log2 > 0 && (kVec<O> << (z.lanes_log2 - 1)) >= a.width) --z.lanes_log2;

    Pass p{};
    p.n = a.n;
    p.vocab = a.vocab;
    p.counts = static_cast<uint32_t*>(sort);
    const bool fill = !a.accumulate && few_tokens(a.n, a.vocab);
    p.occurs = occurs;
    p.clear = !a.accumulate && !fill;
    if (a.n > 0) {
        int last = 1;
        const hipError_t e = own_sort(a.n) ? sort_tokens<O>(a, p, keys, at, z, fill, &last, stream)
                                           : sort_many_tokens(a, p, keys, at, sort, stream);
        if (e != hipSuccess) return e;
        s.keys = keys[last];
        s.at = at[last];
        z.occurs = p.clear ? occurs : nullptr;
    }
    z.first = z.last;   // what the sort's launches did not fill
    z.last = a.accumulate ? z.first : a.vocab;   // nothing, where all of them were
    const Lanes l = lanes_of(up(a.width, kVec<T>));
    s.chunks = l.chunks;
    return l.lanes == 4 ? sum_tokens<T, O, 4>(a, s, z, stream) : l.lanes == 16 ? sum_tokens<T, O, 16>(a, s, z, stream)
                                                                             : sum_tokens<T, O, kWave>(a, s, z, stream);
}

}  // namespace

hipError_t launch_embed(int elem_type, const EmbedArgs& a, hipStream_t stream) {
    if (a.n == 0) return hipSuccess;
    // with scale 1 the rows are copied bit by bit, whatever they hold
    if (a.scale == 1.0f) return elem_type == RS_ELEM_F32 ? embed_of<float, false>(a, stream) : embed_of<_Float16, false>(a, stream);
    switch (elem_type) {
        case RS_ELEM_F32: return embed_of<float, true>(a, stream);
        case RS_ELEM_F16: return embed_of<_Float16, true>(a, stream);
        default: return embed_of<__bf16, true>(a, stream);
    }
}

size_t embed_grad_temp_bytes(int elem_type, uint64_t n, uint32_t vocab, uint32_t width) {
    return Temp(n, vocab, width, elem_type == RS_ELEM_F32 ? kVec<float> : kVec<__bf16>).bytes();
}

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
