// choices.hip -- a router's rows brought into the order of their experts, and
// summed back by their weights, with the gradients of both.
//
// A wave moves a chunk of 64 vectors of 16 bytes of one row.
#include "internal.hpp"
#include "rows_common.hpp"

namespace rs {

namespace {

constexpr int kMoveBlock = 256;
constexpr int kMoveWaves = kMoveBlock / kWave;

// Elements of a 16-byte vector.
template <class T>
constexpr int kVec = 16 / sizeof(T);

// y_i = w_c x_t, c = order_i, t = c / top_k: a wave for each chunk of a position's row.
template <class T, bool WEIGHTS>
__global__ __launch_bounds__(kMoveBlock) void gather_kernel(GatherArgs a, uint32_t chunks) {
    constexpr int V = kVec<T>;
    const uint64_t unit = static_cast<uint64_t>(block_id()) * kMoveWaves + threadIdx.x / kWave;
    const uint64_t i = unit / chunks;
    const uint32_t col = static_cast<uint32_t>(unit % chunks) * (kWave * V) + lane_id() * V;
    if (i >= a.room || col >= a.width) return;
    const uint32_t c = a.order[i];
    const uint32_t left = a.width - col;
    const bool real = c < a.rows * a.top_k;
    const T* from = static_cast<const T*>(a.x) + (real ? c / a.top_k : 0u) * a.x_stride + col;
    T* to = static_cast<T*>(a.y) + i * a.y_stride + col;
    if (WEIGHTS) {
        float v[V] = {};
        if (real) {
            load_some<V>(from, left, 0.0f, v);
            const float w = a.weights[c];
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] *= w;
        }
        store_some<V>(to, left, v);
    } else {
        copy_some<V>(from, real, to, left);
    }
}

// A block for each row: out_t = sum of w y over the row's choices, dots_tj = x_t y.
template <class T, bool WEIGHTS, bool OUT, bool DOTS>
__global__ __launch_bounds__(kMoveBlock) void combine_kernel(CombineArgs a) {
    constexpr int V = kVec<T>;
    __shared__ float s_dots[kMoveWaves][RS_MAX_TOP_K];
    const uint32_t t = block_id();
    if (t >= a.rows) return;
    const uint32_t wave = threadIdx.x / kWave, lane = lane_id();
    if (DOTS) {
        s_dots[wave][lane] = 0.0f;
        wave_fence();
    }
    const uint32_t* place = a.place + static_cast<uint64_t>(t) * a.top_k;
    for (uint32_t col = threadIdx.x * V; col - lane * V < a.width; col += kMoveBlock * V) {
        const uint32_t left = col < a.width ? a.width - col : 0u;
        float sum[V], x[V];
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] = x[e] = 0.0f;
        if (DOTS) load_some<V>(static_cast<const T*>(a.x) + t * a.x_stride + col, left, 0.0f, x);
        for (uint32_t j = 0; j < a.top_k; ++j) {
            const uint32_t p = place[j];
            if (p >= a.room) continue;
            float y[V];
            load_some<V>(static_cast<const T*>(a.y) + p * a.y_stride + col, left, 0.0f, y);
            if (OUT) {
                const float w = WEIGHTS ? a.weights[static_cast<uint64_t>(t) * a.top_k + j] : 1.0f;
#pragma unroll
                for (int e = 0; e < V; ++e) sum[e] = WEIGHTS ? fmaf(w, y[e], sum[e]) : sum[e] + y[e];
            }
            if (DOTS) {
                float dot = 0.0f;
#pragma unroll
                for (int e = 0; e < V; ++e) dot = fmaf(x[e], y[e], dot);
                dot = lanes_sum(dot);
                if (lane == 0) s_dots[wave][j] += dot;
            }
        }
        if (OUT) store_some<V>(static_cast<T*>(a.out) + t * a.out_stride + col, left, sum);
    }
    if (DOTS) {
        __syncthreads();
        if (threadIdx.x < a.top_k) {
            float dot = 0.0f;
#pragma unroll
            for (int w = 0; w < kMoveWaves; ++w) dot += s_dots[w][threadIdx.x];
            a.dots[static_cast<uint64_t>(t) * a.top_k + threadIdx.x] = dot;
        }
    }
}

template <class T>
hipError_t gather_of(const GatherArgs& a, hipStream_t stream) {
    const uint32_t chunks = (a.width + kWave * kVec<T> - 1) / (kWave * kVec<T>);
    const dim3 grid = many_blocks((static_cast<uint64_t>(a.room) * chunks + kMoveWaves - 1) / kMoveWaves);
    timing_before(stream, RS_KERNEL_GATHER);
    if (a.weights) gather_kernel<T, true><<<grid, kMoveBlock, 0, stream>>>(a, chunks);
    else gather_kernel<T, false><<<grid, kMoveBlock, 0, stream>>>(a, chunks);
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

template <class T>
hipError_t combine_of(const CombineArgs& a, hipStream_t stream) {
    const auto kernel = !a.dots ? (a.weights ? combine_kernel<T, true, true, false> : combine_kernel<T, false, true, false>)
                        : a.out ? combine_kernel<T, true, true, true>
                                : combine_kernel<T, true, false, true>;
    timing_before(stream, RS_KERNEL_COMBINE);
    kernel<<<many_blocks(a.rows), kMoveBlock, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

}  // namespace

hipError_t launch_gather(int elem_type, const GatherArgs& a, hipStream_t stream) {
    if (a.room == 0) return hipSuccess;
    switch (elem_type) {
        case RS_ELEM_F32: return gather_of<float>(a, stream);
        case RS_ELEM_F16: return gather_of<_Float16>(a, stream);
        default: return gather_of<__bf16>(a, stream);
    }
}

hipError_t launch_combine(int elem_type, const CombineArgs& a, hipStream_t stream) {
    if (a.rows == 0) return hipSuccess;
    switch (elem_type) {
        case RS_ELEM_F32: return combine_of<float>(a, stream);
        case RS_ELEM_F16: return combine_of<_Float16>(a, stream);
        default: return combine_of<__bf16>(a, stream);
    }
}

}  // namespace rs
