// choices.hip -- a router's rows brought into the order of their experts, and
// summed back by their weights, with the gradients of both:
//   y_i = w_c x_t (c = order_i, t = c / top_k), 0 without a choice;
//   out_t = sum over j of w_tj y_(place_tj); products x_t y_(place_tj).
//
// The row of a token is read once: a wave takes a part of it and writes it to all
// its choices' positions, or sums its choices' rows, eight in flight.  (A wave for
// each position instead reads a row top_k times, from the caches: 333 us for 131072
// choices of 4096 bf16, where a wave each row in an earlier form took 300.)  A choice's
// wave writes a position if order and place name each other there, waves behind look
// for the other positions; so each is written once, as order has it, whatever place
// holds.  Sums and products are f32 in the order of j, products by lanes and then
// waves: nothing depends on the order in which blocks run.
//
// What bounds it is memory: 16384 rows with 8 choices in 163584 positions of 4096
// bf16 take 280 us to gather (5.3 TB/s; writes scattered over 256 segments reach 5.6
// without anything else), 203 to combine (5.8 TB/s); 8192 with 6 of 2048 f16 46 to combine
// and 100 for the gradients (4.5 TB/s).
#include "internal.hpp"
#include "move_common.hpp"

namespace rs {

namespace {

// Rows of up to kNarrow vectors share a wave.  32768 rows with 4 choices, sharing against
// a wave each: of 16 vectors 11.9 us and 13.5 to gather, 8.5 and 11.9 to combine, 20 + 11
// and 25 + 19 for the gradients; of 32 vectors 21.0 and 18.3, 14.9 and 15.0, 40 + 21
// and 35 + 24.
constexpr uint32_t kNarrow = 32;

// ---- wide rows --------------------------------------------------------------------

// The rows of positions that the wave of their choice does not write: zeros
// where there is no choice, and the row itself where place has another position.
template <class T, int U, bool WEIGHTS>
__device__ __forceinline__ void fill_rows(const GatherArgs& a, uint32_t unit, uint32_t parts, uint32_t each) {
    const uint32_t lane = lane_id();
    const uint32_t part = unit % parts;
    const uint32_t i = unit / parts * each + lane;
    const bool here = lane < each && i < a.room;
    const uint32_t c = here ? a.order[i] : 0u;
    const bool real = c < a.rows * a.top_k;
    uint64_t todo = ballot(here && !(real && a.place[c] == i));
    const RowPart<T, U> row(part, a.width);
    while (todo) {
        const uint32_t l = __builtin_ctzll(todo);
        todo &= todo - 1;
        const uint32_t cl = lane_value(c, l);
        typename RowPart<T, U>::Vec r[U] = {};
        if (cl < a.rows * a.top_k) {
            row.load(static_cast<const T*>(a.x) + cl / a.top_k * a.x_stride, r);
            if (WEIGHTS) {
#pragma unroll
                for (int u = 0; u < U; ++u) r[u] = scaled<T>(r[u], a.weights[cl]);
            }
        }
        row.store(static_cast<T*>(a.y) + (unit / parts * each + l) * a.y_stride, r);
    }
}

// A choice's position, and whether the order has it there.
__device__ __forceinline__ bool owns(const uint32_t* order, uint32_t room, uint32_t p, uint32_t c) {
    return p < room && order[p] == c;
}

// A wave for each part of a row, which it reads once and writes to all its
// choices' positions; the waves behind write the other positions, `each` a wave (in
// front of the rows' waves 131072 choices in 163584 positions of 4096 bf16 took 297 us for 282).
template <class T, int U, bool WEIGHTS>
__global__ __launch_bounds__(kMoveBlock) void gather_kernel(GatherArgs a, uint32_t parts, uint32_t each) {
    const uint32_t unit = block_id() * kMoveWaves + wave_id();
    const uint32_t rows = a.rows * parts;   // waves
    if (unit >= rows) return fill_rows<T, U, WEIGHTS>(a, unit - rows, parts, each);
    const uint32_t t = unit / parts, part = unit % parts;
    const uint32_t lane = lane_id();
    const uint32_t c = t * a.top_k + lane;
    const RowPart<T, U> row(part, a.width);
    typename RowPart<T, U>::Vec x[U];
    row.load(static_cast<const T*>(a.x) + t * a.x_stride, x);
    uint32_t p = lane < a.top_k ? a.place[c] : ~0u;
    float w = WEIGHTS && lane < a.top_k ? a.weights[c] : 0.0f;
    arrived(p, w);
    uint64_t todo = ballot(owns(a.order, a.room, p, c));
    while (todo) {
        const uint32_t l = __builtin_ctzll(todo);
        todo &= todo - 1;
        T* to = static_cast<T*>(a.y) + lane_value(p, l) * a.y_stride;
        if (WEIGHTS) {
            typename RowPart<T, U>::Vec r[U];
            const float wl = lane_value(w, l);
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = scaled<T>(x[u], wl);
            row.store(to, r);
        } else {
            row.store(to, x);
        }
    }
}

constexpr int kBatch = 8;   // choices whose rows are in flight together

// A wave for each 64 vectors of a row: the sum of its choices' rows there.
template <class T, bool WEIGHTS, bool ONCE>
__global__ __launch_bounds__(kMoveBlock) void combine_kernel(CombineArgs a, uint32_t parts) {
    using Row = RowPart<T, 1>;
    constexpr int V = kVec<T>;
    const uint32_t unit = block_id() * kMoveWaves + wave_id();
    const uint32_t t = unit / parts;
    if (t >= a.rows) return;
    const uint32_t lane = lane_id();
    const Row row(unit % parts, a.width);
    uint32_t p = lane < a.top_k ? a.place[t * a.top_k + lane] : ~0u;
    float w = WEIGHTS && lane < a.top_k ? a.weights[t * a.top_k + lane] : 1.0f;
    arrived(p, w);
    float sum[V] = {};
    for (uint64_t todo = ballot(p < a.room); todo != 0;) {
        typename Row::Vec r[kBatch][1];
        float wl[kBatch];
        uint32_t n = 0;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (todo == 0) break;
            const uint32_t l = __builtin_ctzll(todo);
            todo &= todo - 1;
            wl[b] = lane_value(w, l);
            row.template load<ONCE>(static_cast<const T*>(a.y) + lane_value(p, l) * a.y_stride, r[b]);
            ++n;
        }
#pragma unroll
        for (uint32_t b = 0; b < kBatch; ++b) {
            if (b >= n) break;
            float y[V];
            widen<T>(r[b][0], y);
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] = WEIGHTS ? fmaf(wl[b], y[e], sum[e]) : sum[e] + y[e];
        }
    }
    const typename Row::Vec out[1] = {narrow<T>(sum)};
    row.store(static_cast<T*>(a.out) + t * a.out_stride, out);
}

// Gradients, WAVES waves a row: the products of x_t with the rows of y at its
// choices, and beside them the sum of those rows by their weights (SUM), or x_t
// times each weight at its choices' positions in g.y.  MANY: more than kBatch choices a row.
template <class T, int WAVES, bool SUM, bool MANY>
__global__ __launch_bounds__(kMoveBlock, 4) void products_kernel(CombineArgs a, GatherArgs g, uint32_t fill,
                                                                 uint32_t fill_parts, uint32_t each) {
    using Row = RowPart<T, 1>;
    constexpr int V = kVec<T>;
    __shared__ float s_dots[kMoveWaves][RS_MAX_TOP_K];
    const uint32_t wave = wave_id(), lane = lane_id();
    if (!SUM && block_id() < fill) return fill_rows<T, 4, true>(g, block_id() * kMoveWaves + wave, fill_parts, each);
    const uint32_t t = ((block_id() - fill) * kMoveWaves + wave) / WAVES;
    const bool real = t < a.rows;
    s_dots[wave][lane] = 0.0f;
    wave_fence();
    if (real) {
        const uint32_t c = t * a.top_k + lane;
        uint32_t p = lane < a.top_k ? a.place[c] : ~0u;
        float w = lane < a.top_k ? a.weights[c] : 0.0f;
        arrived(p, w);
        const uint64_t valid = ballot(p < a.room);
        const uint64_t owned = SUM ? 0 : ballot(owns(g.order, g.room, p, c));
        const uint32_t steps = (a.width + kWave * V - 1) / (kWave * V);
        const T* x_row = static_cast<const T*>(a.x) + t * a.x_stride;
        float dot[kBatch] = {};   // of the valid choices, in order
        for (uint32_t s = wave % WAVES; s < steps; s += WAVES) {
            const Row row(s, a.width);
            const typename Row::Vec own = row.own_bits(s, 0);
            typename Row::Vec xr[1];
            row.load(x_row, xr);
            float x[V], sum[V] = {};
            uint64_t todo = valid;
            do {   // once without MANY, so that the load of x goes out with the others
                typename Row::Vec r[kBatch][1];
                uint32_t l[kBatch], n = 0;
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    if (todo == 0) break;
                    l[b] = __builtin_ctzll(todo);
                    todo &= todo - 1;
                    row.load(static_cast<const T*>(a.y) + lane_value(p, l[b]) * a.y_stride, r[b]);
                    ++n;
                }
                widen<T>(xr[0] & own, x);
#pragma unroll
                for (uint32_t b = 0; b < kBatch; ++b) {
                    if (b >= n) break;
                    float y[V];
                    const float wl = lane_value(w, l[b]);
                    if (SUM) {
                        widen<T>(r[b][0], y);
#pragma unroll
                        for (uint32_t e = 0; e < V; ++e) sum[e] = fmaf(wl, y[e], sum[e]);
                    }
                    widen<T>(r[b][0] & own, y);
#pragma unroll
                    for (uint32_t e = 0; e < V; ++e) dot[b] = fmaf(x[e], y[e], dot[b]);
                }
                if (MANY) {
#pragma unroll
                    for (uint32_t b = 0; b < kBatch; ++b) {
                        if (b >= n) break;
                        const float d = lanes_sum(dot[b]);
                        if (lane == 0) s_dots[wave][l[b]] += d;
                        dot[b] = 0.0f;
                    }
                }
            } while (MANY && todo != 0);
            if (SUM) {
                const typename Row::Vec v[1] = {narrow<T>(sum)};
                row.store(static_cast<T*>(a.out) + t * a.out_stride, v);
            } else {
                for (uint64_t own_places = owned; own_places != 0; own_places &= own_places - 1) {
                    const uint32_t b = __builtin_ctzll(own_places);
                    const typename Row::Vec v[1] = {scaled<T>(xr[0], lane_value(w, b))};
                    row.store(static_cast<T*>(g.y) + lane_value(p, b) * g.y_stride, v);
                }
            }
        }
        if (!MANY) {
            uint64_t todo = valid;
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (todo == 0) break;
                const float d = lanes_sum(dot[b]);
                if (lane == 0) s_dots[wave][__builtin_ctzll(todo)] = d;
                todo &= todo - 1;
            }
        }
    }
    if (WAVES > 1) __syncthreads();
    else wave_fence();
    if (real && wave % WAVES == 0 && lane < a.top_k) {
        float d = 0.0f;
#pragma unroll
        for (int v = 0; v < WAVES; ++v) d += s_dots[wave + v][lane];
        a.dots[t * a.top_k + lane] = d;
    }
}

// ---- narrow rows: L lanes a row -----------------------------------------------------

constexpr int kRowsEach = 4;   // positions of a group of lanes

template <class T, int L, bool WEIGHTS>
__device__ __forceinline__ void gather_narrow(const GatherArgs& a, uint32_t block) {
    constexpr int V = kVec<T>;
    constexpr uint32_t kGroups = kMoveBlock / L;
    const uint32_t col = threadIdx.x % L * V;
    if (col >= a.width) return;
    const uint32_t left = a.width - col;
    uint32_t c[kRowsEach];
    uint64_t i = static_cast<uint64_t>(block) * (kGroups * kRowsEach) + threadIdx.x / L;
#pragma unroll
    for (int u = 0; u < kRowsEach; ++u) c[u] = i + u * kGroups < a.room ? a.order[i + u * kGroups] : ~0u;
    float v[kRowsEach][V];
#pragma unroll
    for (int u = 0; u < kRowsEach; ++u, i += kGroups) {
        if (i >= a.room) return;
        const bool real = c[u] < a.rows * a.top_k;
        const T* from = static_cast<const T*>(a.x) + (real ? c[u] / a.top_k : 0u) * a.x_stride + col;
        T* to = static_cast<T*>(a.y) + i * a.y_stride + col;
        if (WEIGHTS) {
#pragma unroll
            for (int e = 0; e < V; ++e) v[u][e] = 0.0f;
            if (real) {
                load_some<V>(from, left, 0.0f, v[u]);
                const float w = a.weights[c[u]];
#pragma unroll
                for (int e = 0; e < V; ++e) v[u][e] *= w;
            }
            store_some<V>(to, left, v[u]);
        } else {
            copy_some<V>(from, real, to, left);
        }
    }
}

template <class T, int L, bool WEIGHTS, bool OUT, bool DOTS>
__device__ __forceinline__ void combine_narrow(const CombineArgs& a, uint32_t block) {
    constexpr int V = kVec<T>;
    constexpr uint32_t kEach = 4;   // choices in flight
    const uint32_t t = block * (kMoveBlock / L) + threadIdx.x / L;
    if (t >= a.rows) return;
    const uint32_t col = threadIdx.x % L * V;
    const uint32_t left = col < a.width ? a.width - col : 0u;
    float sum[V] = {}, x[V];
    if (DOTS) load_some<V>(static_cast<const T*>(a.x) + t * a.x_stride + col, left, 0.0f, x);
    for (uint32_t j0 = 0; j0 < a.top_k; j0 += kEach) {
        uint32_t p[kEach];
        float w[kEach], y[kEach][V];
#pragma unroll
        for (uint32_t b = 0; b < kEach; ++b) {
            p[b] = j0 + b < a.top_k ? a.place[t * a.top_k + j0 + b] : ~0u;
            w[b] = WEIGHTS && j0 + b < a.top_k ? a.weights[t * a.top_k + j0 + b] : 1.0f;
        }
#pragma unroll
        for (uint32_t b = 0; b < kEach; ++b)
            if (p[b] < a.room) load_some<V>(static_cast<const T*>(a.y) + p[b] * a.y_stride + col, left, 0.0f, y[b]);
#pragma unroll
        for (uint32_t b = 0; b < kEach; ++b) {
            float dot = 0.0f;
            if (p[b] < a.room) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (OUT) sum[e] = WEIGHTS ? fmaf(w[b], y[b][e], sum[e]) : sum[e] + y[b][e];
                    if (DOTS) dot = fmaf(x[e], y[b][e], dot);
                }
            }
            if (DOTS) {
                dot = lanes_sum<L>(dot);
                if (threadIdx.x % L == 0 && j0 + b < a.top_k) a.dots[t * a.top_k + j0 + b] = dot;
            }
        }
    }
    if (OUT) store_some<V>(static_cast<T*>(a.out) + t * a.out_stride + col, left, sum);
}

template <class T, int L, bool WEIGHTS>
__global__ __launch_bounds__(kMoveBlock) void gather_narrow_kernel(GatherArgs a) {
    gather_narrow<T, L, WEIGHTS>(a, block_id());
}
template <class T, int L, bool WEIGHTS>
__global__ __launch_bounds__(kMoveBlock) void combine_narrow_kernel(CombineArgs a) {
    combine_narrow<T, L, WEIGHTS, true, false>(a, block_id());
}
template <class T, int L, bool SUM>
__global__ __launch_bounds__(kMoveBlock) void products_narrow_kernel(CombineArgs a, GatherArgs g, uint32_t fill) {
    if (!SUM && block_id() < fill) gather_narrow<T, L, true>(g, block_id());
    else combine_narrow<T, L, true, SUM, true>(a, block_id() - fill);
}

// ---- launches ---------------------------------------------------------------------

template <class Launch>
hipError_t timed(int id, hipStream_t stream, Launch launch) {
    timing_before(stream, id);
    launch();
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

// call(whether) as a constant.
template <class Call>
void pick(bool whether, Call call) {
    if (whether) call(std::true_type{});
    else call(std::false_type{});
}

// Positions that a wave fills: few where there is padding, which is all that it
// writes, many where there is none and it only looks.  Gathering, whose filling is
// behind the rows: with padding, 131072 choices in 163584 positions of 4096 bf16 281 us with
// 4 and 284 with 16, 16384 in 16504 of 1024 f16 10.8 and 13.4, 2000 in 2112 of 2048 bf16 4.3 and 6.1;
// without, 15005 of 1001 f32 13.5 and 13.0, 24000 of 1024 f16 13.3 and 12.9.
uint32_t fill_each(uint64_t room, uint64_t choices) { return room > choices ? 4 : 16; }
// In front of the products (and with the combining, which is the same), few only where
// much is padding: 80000 choices in 80448 positions of 512 bf16 58.7 us with 4 and 56.2 with 16,
// 24000 in 24120 of 1024 41.7 and 40.8; 2000 in 6032 of 2048 12.1 and 14.1, 16000 in 22336 of
// 1001 f32 54.3 and 54.2, 65536 in 98048 of 2048 bf16 207 and 205.
uint32_t fill_each_in_front(uint64_t room, uint64_t choices) { return fill_each(room, choices + choices / 16); }

// call(lanes a row) of a narrow row.
template <class Call>
hipError_t by_lanes(uint32_t vectors, Call call) {
    if (vectors <= 4) return call(std::integral_constant<int, 4>{});
    if (vectors <= 16) return call(std::integral_constant<int, 16>{});
    return call(std::integral_constant<int, 32>{});
}

template <class T, bool WEIGHTS>
hipError_t gather_of(const GatherArgs& a, hipStream_t stream) {
    const uint32_t vectors = static_cast<uint32_t>(up(a.width, kVec<T>));
    if (vectors <= kNarrow)
        return by_lanes(vectors, [&](auto lanes) {
            constexpr int L = decltype(lanes)::value;
            return timed(RS_KERNEL_GATHER, stream, [&] {
                gather_narrow_kernel<T, L, WEIGHTS><<<many_blocks(up(a.room, kMoveBlock / L * kRowsEach)), kMoveBlock, 0, stream>>>(a);
            });
        });
    const Split s = split_rows(vectors, a.rows, 4);
    const uint32_t each = fill_each(a.room, static_cast<uint64_t>(a.rows) * a.top_k);
    const dim3 grid = many_blocks(up((a.rows + up(a.room, each)) * s.parts, kMoveWaves));
    return timed(RS_KERNEL_GATHER, stream, [&] {
        const auto kernel = s.unroll == 1 ? gather_kernel<T, 1, WEIGHTS> : s.unroll == 2 ? gather_kernel<T, 2, WEIGHTS>
                                                                                         : gather_kernel<T, 4, WEIGHTS>;
        kernel<<<grid, kMoveBlock, 0, stream>>>(a, s.parts, each);
    });
}

template <class T, bool WEIGHTS>
hipError_t combine_of(const CombineArgs& a, hipStream_t stream) {
    const uint32_t vectors = static_cast<uint32_t>(up(a.width, kVec<T>));
    if (vectors <= kNarrow)
        return by_lanes(vectors, [&](auto lanes) {
            constexpr int L = decltype(lanes)::value;
            return timed(RS_KERNEL_COMBINE, stream, [&] {
                combine_narrow_kernel<T, L, WEIGHTS><<<many_blocks(up(a.rows, kMoveBlock / L)), kMoveBlock, 0, stream>>>(a);
            });
        });
    const uint32_t parts = static_cast<uint32_t>(up(vectors, kWave));
    return timed(RS_KERNEL_COMBINE, stream, [&] {
        pick(large(static_cast<uint64_t>(a.rows) * a.top_k * a.width * sizeof(T)), [&](auto once) {
            constexpr bool ONCE = decltype(once)::value;
            combine_kernel<T, WEIGHTS, ONCE><<<many_blocks(up(static_cast<uint64_t>(a.rows) * parts, kMoveWaves)), kMoveBlock, 0, stream>>>(a, parts);
        });
    });
}

template <class T, bool SUM>
hipError_t products_of(const CombineArgs& a, const GatherArgs& g, hipStream_t stream) {
    const uint32_t vectors = static_cast<uint32_t>(up(a.width, kVec<T>));
    if (vectors <= kNarrow)
        return by_lanes(vectors, [&](auto lanes) {
            constexpr int L = decltype(lanes)::value;
            const uint32_t fill = SUM ? 0 : static_cast<uint32_t>(up(g.room, kMoveBlock / L * kRowsEach));
            return timed(RS_KERNEL_COMBINE, stream, [&] {
                products_narrow_kernel<T, L, SUM><<<many_blocks(fill + up(a.rows, kMoveBlock / L)), kMoveBlock, 0, stream>>>(a, g, fill);
            });
        });
    const uint32_t waves = vectors <= kWave ? 1 : vectors <= 2 * kWave ? 2 : 4;   // of a row; 8192 rows of 256 vectors: 146 us with 4, 160 with 1
    const uint32_t parts = static_cast<uint32_t>(up(vectors, 4 * kWave));
    const uint32_t each = fill_each_in_front(g.room, static_cast<uint64_t>(a.rows) * a.top_k);
    const uint32_t fill = SUM ? 0 : static_cast<uint32_t>(up(up(g.room, each) * parts, kMoveWaves));
    return timed(RS_KERNEL_COMBINE, stream, [&] {
        pick(a.top_k > kBatch, [&](auto many) {
            constexpr bool MANY = decltype(many)::value;
            const auto kernel = waves == 1 ? products_kernel<T, 1, SUM, MANY> : waves == 2 ? products_kernel<T, 2, SUM, MANY>
                                                                                           : products_kernel<T, 4, SUM, MANY>;
            kernel<<<many_blocks(fill + up(uint64_t{a.rows} * waves, kMoveWaves)), kMoveBlock, 0, stream>>>(a, g, fill, parts, each);
        });
    });
}

template <class T>
hipError_t combine_any(const CombineArgs& a, hipStream_t stream) {
    if (a.dots) return products_of<T, true>(a, GatherArgs{}, stream);
    return a.weights ? combine_of<T, true>(a, stream) : combine_of<T, false>(a, stream);
}

}  // namespace

hipError_t launch_gather(int elem_type, const GatherArgs& a, hipStream_t stream) {
    if (a.room == 0) return hipSuccess;
    // without weights the rows are copied bit by bit, whatever they hold
    if (!a.weights) return elem_type == RS_ELEM_F32 ? gather_of<float, false>(a, stream) : gather_of<_Float16, false>(a, stream);
    switch (elem_type) {
        case RS_ELEM_F32: return gather_of<float, true>(a, stream);
        case RS_ELEM_F16: return gather_of<_Float16, true>(a, stream);
        default: return gather_of<__bf16, true>(a, stream);
    }
}

hipError_t launch_combine(int elem_type, const CombineArgs& a, hipStream_t stream) {
    if (a.rows == 0) return hipSuccess;
    switch (elem_type) {
        case RS_ELEM_F32: return combine_any<float>(a, stream);
        case RS_ELEM_F16: return combine_any<_Float16>(a, stream);
        default: return combine_any<__bf16>(a, stream);
    }
}

hipError_t launch_combine_grad(int elem_type, const CombineArgs& a, const GatherArgs& g, hipStream_t stream) {
    if (a.rows == 0 && g.room == 0) return hipSuccess;
    switch (elem_type) {
        case RS_ELEM_F32: return products_of<float, false>(a, g, stream);
        case RS_ELEM_F16: return products_of<_Float16, false>(a, g, stream);
        default: return products_of<__bf16, false>(a, g, stream);
    }
}

}  // namespace rs
