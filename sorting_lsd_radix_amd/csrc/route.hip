// route.hip -- a router's choices: the best experts of each row of scores,
// their weights, and the weights' gradient.
//
// One wave works on one row.  The row's scores are read once into registers:
// lane l holds experts l * V .. l * V + V - 1, so that (lane, slot) is the
// order of the experts and a tie between lanes goes to the lower one.
#include "internal.hpp"
#include "rows_common.hpp"

namespace rs {

namespace {

constexpr int kRouteWaves = 4;                      // rows of a block

// The largest of the lanes' 64-bit patterns, and the lowest lane that has it.
__device__ __forceinline__ uint64_t wave_best(uint64_t k, uint32_t* lane_of) {
    uint64_t b = k;
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) {
        const uint64_t o = __shfl_xor(b, off, kWave);
        b = o > b ? o : b;
    }
    *lane_of = static_cast<uint32_t>(__builtin_ctzll(ballot(k == b)));
    return b;
}

template <int ELEM, int V, bool SIGMOID>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_kernel(RouteArgs a) {
    using T = typename Elem<ELEM>::T;
    __shared__ double s_score[kRouteWaves][RS_MAX_EXPERTS];
    __shared__ float s_x[kRouteWaves][RS_MAX_EXPERTS];
    const uint32_t wave = threadIdx.x / kWave;
    const uint32_t lane = threadIdx.x & (kWave - 1);
    const uint32_t row = block_id() * kRouteWaves + wave;
    if (row >= a.rows) return;
    const T* in = static_cast<const T*>(a.scores) + row * a.row_stride;

    float x[V];
    float m = -__builtin_huge_valf();
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t e = lane * V + j;
        x[j] = e < a.experts ? static_cast<float>(in[e]) : -__builtin_huge_valf();
        m = fmaxf(m, x[j]);
    }
    m = lanes_max(m);
    const bool empty = m == -__builtin_huge_valf();   // of softmax rows with NaN too: the sum is NaN then
    double total = 1.0;
    if (!SIGMOID) {
        double mine = 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (lane * V + j < a.experts)
                mine += (empty && x[j] == x[j]) ? 0.0 : exp(static_cast<double>(x[j]) - static_cast<double>(m));
        total = lanes_sum(mine);
    }
    auto prob = [&](float v) -> double {
        if (SIGMOID) return 1.0 / (1.0 + exp(-static_cast<double>(v)));
        if (empty && total == 0.0) return 0.0;
        return exp(static_cast<double>(v) - static_cast<double>(m)) / total;
    };

    uint64_t key[V];
    const bool by_p = a.bias != nullptr;
    const bool group_p = a.groups > 1 && (by_p || a.group_best == 2);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t e = lane * V + j;
        key[j] = 0;
        if (e < a.experts) {
            const bool masked = !(x[j] > -__builtin_huge_valf());
            double s = x[j];
            if (by_p) s = masked ? -__builtin_huge_val() : prob(x[j]) + static_cast<double>(a.bias[e]);
            key[j] = order64_masked(s);
            if (a.groups > 1) s_score[wave][e] = group_p && !by_p ? (masked ? -__builtin_huge_val() : prob(x[j])) : s;
            s_x[wave][e] = x[j];
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");

    if (a.groups > 1) {
        const uint32_t size = a.experts / a.groups;
        uint64_t gkey = 0;
        if (lane < a.groups) {
            double best = -__builtin_huge_val(), next = -__builtin_huge_val();
            for (uint32_t i = 0; i < size; ++i) {
                const double s = s_score[wave][lane * size + i];
                if (s > best) {
                    next = best;
                    best = s;
                } else if (s > next) {
                    next = s;
                }
            }
            if (a.group_best == 2 && next > -__builtin_huge_val()) best += next;
            gkey = order64_masked(best);
        }
        uint64_t kept = 0;
        for (uint32_t r = 0; r < a.top_groups; ++r) {
            uint32_t g;
            wave_best(gkey, &g);
            kept |= 1ull << g;
            if (lane == g) gkey = 0;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t e = lane * V + j;
            if (e < a.experts && !((kept >> (e / size)) & 1ull)) key[j] = 0;
        }
    }

    uint32_t chosen = 0;   // lane r holds the r-th choice
    for (uint32_t r = 0; r < a.top_k; ++r) {
        uint64_t mine = 0;
        uint32_t slot = 0;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (key[j] > mine) {
                mine = key[j];
                slot = j;
            }
        uint32_t from;
        wave_best(mine, &from);
        const uint32_t e = __shfl(lane * V + slot, from, kWave);
        if (lane == from) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j == static_cast<int>(slot)) key[j] = 0;
        }
        if (lane == r) chosen = e;
    }

    const bool mine = lane < a.top_k;
    const double p = mine ? prob(s_x[wave][chosen]) : 0.0;
    double w = static_cast<double>(a.scale) * p;
    if (a.renormalize) {
        const double sum = lanes_sum(p);
        w = sum == 0.0 ? 0.0 : w / sum;
    }
    if (mine) {
        const uint64_t at = static_cast<uint64_t>(row) * a.top_k + lane;
        a.ids[at] = chosen;
        a.weights[at] = static_cast<float>(w);
    }
}

template <int ELEM, int V, bool SIGMOID>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_grad_kernel(RouteGradArgs a) {
    using T = typename Elem<ELEM>::T;
    const uint32_t wave = threadIdx.x / kWave;
    const uint32_t lane = threadIdx.x & (kWave - 1);
    const uint32_t row = block_id() * kRouteWaves + wave;
    if (row >= a.rows) return;
    const T* in = static_cast<const T*>(a.scores) + row * a.row_stride;
    T* out = static_cast<T*>(a.dscores) + row * a.dscores_stride;

    const bool mine = lane < a.top_k;
    const uint64_t at = static_cast<uint64_t>(row) * a.top_k + lane;
    const uint32_t id = mine ? a.ids[at] : 0xFFFFFFFFu;
    const float w = mine ? a.weights[at] : 0.0f;
    const float dw = mine ? a.dweights[at] : 0.0f;
    const float d = lanes_sum(dw * w);
    float part = w * (a.renormalize ? dw - d / a.scale : dw);   // the choice's own term

    float dx[V];
#pragma unroll
    for (int j = 0; j < V; ++j) dx[j] = 0.0f;
    if (SIGMOID) {
        if (id < a.experts) part *= 1.0f / (1.0f + expf(static_cast<float>(in[id])));
    } else if (!a.renormalize) {
        float x[V];
        float m = -__builtin_huge_valf();
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t e = lane * V + j;
            x[j] = e < a.experts ? static_cast<float>(in[e]) : -__builtin_huge_valf();
            m = fmaxf(m, x[j]);
        }
        m = lanes_max(m);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (lane * V + j < a.experts) {
                x[j] = expf(x[j] - m);
                sum += x[j];
            }
        sum = lanes_sum(sum);
        const bool empty = m == -__builtin_huge_valf();   // p = 0 (and d = 0, or NaN where the weights are)
#pragma unroll
        for (int j = 0; j < V; ++j) dx[j] = -(empty ? 0.0f : x[j] / sum) * d;
    }
    for (uint32_t r = 0; r < a.top_k; ++r) {
        const uint32_t e = __shfl(id, r, kWave);
        const float g = __shfl(part, r, kWave);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e == lane * V + j) dx[j] += g;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t e = lane * V + j;
        if (e < a.experts) out[e] = static_cast<T>(dx[j]);
    }
}

template <int ELEM, int V>
hipError_t route_shape(const RouteArgs& a, hipStream_t stream) {
    const uint32_t blocks = (a.rows + kRouteWaves - 1) / kRouteWaves;
    timing_before(stream, RS_KERNEL_ROUTE);
    if (a.sigmoid)
        route_kernel<ELEM, V, true><<<many_blocks(blocks), kRouteWaves * kWave, 0, stream>>>(a);
    else
        route_kernel<ELEM, V, false><<<many_blocks(blocks), kRouteWaves * kWave, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

template <int ELEM, int V>
hipError_t grad_shape(const RouteGradArgs& a, hipStream_t stream) {
    const uint32_t blocks = (a.rows + kRouteWaves - 1) / kRouteWaves;
    timing_before(stream, RS_KERNEL_ROUTE_GRAD);
    if (a.sigmoid)
        route_grad_kernel<ELEM, V, true><<<many_blocks(blocks), kRouteWaves * kWave, 0, stream>>>(a);
    else
        route_grad_kernel<ELEM, V, false><<<many_blocks(blocks), kRouteWaves * kWave, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

template <int ELEM>
hipError_t route_elem(const RouteArgs& a, hipStream_t stream) {
    if (a.experts <= 64) return route_shape<ELEM, 1>(a, stream);
    if (a.experts <= 256) return route_shape<ELEM, 4>(a, stream);
    return route_shape<ELEM, 16>(a, stream);
}

template <int ELEM>
hipError_t grad_elem(const RouteGradArgs& a, hipStream_t stream) {
    if (a.experts <= 64) return grad_shape<ELEM, 1>(a, stream);
    if (a.experts <= 256) return grad_shape<ELEM, 4>(a, stream);
    return grad_shape<ELEM, 16>(a, stream);
}

}  // namespace

hipError_t launch_route(int elem_type, const RouteArgs& a, hipStream_t stream) {
    switch (elem_type) {
    case RS_ELEM_F32: return route_elem<RS_ELEM_F32>(a, stream);
    case RS_ELEM_F16: return route_elem<RS_ELEM_F16>(a, stream);
    default: return route_elem<RS_ELEM_BF16>(a, stream);
    }
}

hipError_t launch_route_grad(int elem_type, const RouteGradArgs& a, hipStream_t stream) {
    switch (elem_type) {
    case RS_ELEM_F32: return grad_elem<RS_ELEM_F32>(a, stream);
    case RS_ELEM_F16: return grad_elem<RS_ELEM_F16>(a, stream);
    default: return grad_elem<RS_ELEM_BF16>(a, stream);
    }
}

}  // namespace rs
