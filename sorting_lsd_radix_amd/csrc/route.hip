// route.hip -- a router's choices: the best experts of each row of scores,
// their weights, and the weights' gradient.
//
// A row is the work of L lanes (16, 32 or 64) of a wave, which so works on 64 /
// L rows at once: lane l of a row holds its experts l V .. l V + V - 1 in
// registers, read once.  The reductions over a row are then log2(L) lane
// exchanges that serve every row of the wave.
//
// The choice is by s in 64 bits (in f32, some of 16384 rows of 256 experts
// choose another expert than the definition's), yet only a row's candidates
// are computed so: s in f32, which is off by at most kOff, leaves out every
// expert that cannot be among the first, and decides which groups are kept
// unless two scores at the border are too near (then the row's s are all taken
// in 64 bits).  64-bit arithmetic for every expert cost 45 us of 32768 rows of
// 512 experts' sigmoids with a bias, against 30 without.  A softmax whose sum is
// needed (with a bias, groups by pairs or weights that stay p) still takes the
// exponential of every expert in 64 bits.
//
// What bounds it: 32768 rows of 512 f32 (67 MB), sigmoid with a bias, take 25-28
// us, 2.4-2.7 TB/s, with the vector units busy in 0.92 of the compute units'
// cycles (790 instructions for the two rows of a wave), softmax with a bias 35;
// 16384 rows of 256 with groups 16-20 us, where a wave's dependent steps count as
// much.  Below some 4096 rows the launch is all.
//
// Slower rows: those with more candidates than a row has lanes, whose choices are
// taken one after the other (equal scores, a mask that leaves fewer lanes than
// top_k, kept groups on fewer lanes than that: 32768 rows of 512, sigmoid with a
// bias, 77, 58 and 90 us), and those whose groups f32 cannot tell apart (equal
// scores in groups by pairs: 139 us, 16384 rows of 256 42).
#include "internal.hpp"
#include "rows_common.hpp"

namespace rs {

namespace {

constexpr int kRouteWaves = 4;

constexpr float kInf = __builtin_huge_valf();

// In 64 bits, s of experts that cannot be chosen and of masked ones (behind
// every other, but a choice where nothing else is left); no s is so low, as
// scores and biases are f32.  In f32 these are NaN and -inf.
constexpr double kExcluded = -__builtin_huge_val();
constexpr double kMasked = -1.7976931348623157e308;

// How far s in f32 may be off: kOff + kOffRel |s|.  p = 1 / (1 + e) has at most
// 4 roundings' worth, 2^-22 (exp2's argument is off by 2^-24 |x log2 e|, which
// moves p by less than p (1 - p) |x| 2^-24 < 2^-26; exp2 and the reciprocal are
// off by 2^-23 relative, the sum by 2^-24); adding the bias 2^-24 |s|.  Twice that.
// A softmax's p has three roundings relative to it, which is less; of a peaked row
// the small p are so taken for nearer to each other than they are, and more
// groups compared in 64 bits (32768 rows of 512 in groups by pairs, scores spread
// by 12 instead of 1.5: 74 us for 53).
constexpr float kOff = 0x1p-21f;
constexpr float kOffRel = 0x1p-23f;

// exp(x): 2^n exp(r) with n = x / ln 2 to nearest and |r| <= ln 2 / 2, exp(r) by
// Taylor's series to r^13 / 13! (the next term is below 2^-57).  Arguments
// beyond +-1100 (infinities among them) give infinity and 0; NaN gives 0.
__device__ __forceinline__ double exp64(double x) {
    x = fmin(fmax(x, -1100.0), 1100.0);
    const double n = rint(x * 1.4426950408889634074);
    double r = fma(n, -0.69314718055994530942, x);
    r = fma(n, -2.3190468138462995584e-17, r);   // ln 2 less its double
    double e = 1.0 / 6227020800.0;
    e = fma(e, r, 1.0 / 479001600.0);
    e = fma(e, r, 1.0 / 39916800.0);
    e = fma(e, r, 1.0 / 3628800.0);
    e = fma(e, r, 1.0 / 362880.0);
    e = fma(e, r, 1.0 / 40320.0);
    e = fma(e, r, 1.0 / 5040.0);
    e = fma(e, r, 1.0 / 720.0);
    e = fma(e, r, 1.0 / 120.0);
    e = fma(e, r, 1.0 / 24.0);
    e = fma(e, r, 1.0 / 6.0);
    e = fma(e, r, 0.5);
    e = fma(e, r, 1.0);
    e = fma(e, r, 1.0);
    return ldexp(e, static_cast<int>(n));
}

// What a row's probabilities are computed with: sigmoid, or softmax with the
// largest score m and the sum of exp relative to it (1 where only ratios are
// wanted), and whether the row has a NaN (softmax: all its p are NaN).
struct Prob {
    bool sigmoid, nan;
    double m, sum;

    __device__ __forceinline__ double operator()(float x) const {
        if (sigmoid) return x != x ? __builtin_nan("") : 1.0 / (1.0 + exp64(-static_cast<double>(x)));
        if (nan || m == __builtin_huge_val()) return __builtin_nan("");
        if (m == -__builtin_huge_val()) return 0.0;
        return exp64(static_cast<double>(x) - m) / sum;
    }
};

// A row's candidates in LDS, at most L.
struct Candidate {
    double s;
    float x;
    uint32_t e;
};

// The best two scores of the group that `p` lanes share, from each lane's two;
// then the group's score into the row's LDS, best_of [groups], and in f32 the
// size of its terms, which its error goes by, behind it.
template <class S>
__device__ __forceinline__ void group_score(const RouteArgs& a, S best, S next, uint32_t sub, uint32_t p, S masked,
                                            S* best_of) {
    for (uint32_t o = 1; o < p; o <<= 1) {
        const S b = __shfl_xor(best, static_cast<int>(o), kWave), n = __shfl_xor(next, static_cast<int>(o), kWave);
        next = fmax(fmax(next, n), fmin(best, b));
        best = fmax(best, b);
    }
    const uint32_t g = sub / p;
    if (g < a.groups && sub == g * p) {
        const bool two = a.group_best == 2 && next > masked;
        S sum = two ? best + next : best;
        if (sizeof(S) == 4) {
            // a sum below f32's range is not a masked group's
            if (best > masked) sum = fmax(sum, S(-3.402823466e38f));
            best_of[a.groups + g] = fabs(best) + (two ? fabs(next) : S(0));
        }
        best_of[g] = sum;
    }
}

// The same from the scores of all experts in the row's LDS, score [experts]: p =
// L / (groups, rounded up to a power of two) lanes share a group.
template <int L, class S>
__device__ __forceinline__ void group_scores(const RouteArgs& a, const S* score, S* best_of, S masked) {
    const uint32_t sub = lane_id() & (L - 1);
    const uint32_t size = a.experts / a.groups;
    uint32_t p = L;
    while (p * a.groups > L) p >>= 1;
    const uint32_t g = sub / p;
    S best = masked, next = masked;
    if (g < a.groups) {
#pragma unroll 4
        for (uint32_t i = sub & (p - 1); i < size; i += p) {
            const S s = score[g * size + i];
            next = fmax(next, fmin(best, s));
            best = fmax(best, s);
        }
    }
    group_score(a, best, next, sub, p, masked, best_of);
}

// The kept groups of the wave's rows, as masks (equal in a row's lanes), from
// the groups' scores best_of [groups] (f32 or 64 bits).  Two f32 scores may be
// off by off + rel * (the size of their terms) together; `unclear` tells whether
// that leaves the row's choice open.
template <int L, class S>
__device__ __forceinline__ uint64_t kept_groups(const RouteArgs& a, const S* best_of, S masked, S off, S rel,
                                                bool* unclear) {
    const uint32_t lane = lane_id();
    const uint32_t sub = lane & (L - 1);
    wave_fence();
    bool kept = false, open = false;
    if (sub < a.groups) {   // groups before this one, and groups that may be
        const S mine = best_of[sub];
        const S size = sizeof(S) == 4 ? best_of[a.groups + sub] : S(0);
        uint32_t before = 0, near = 0;
#pragma unroll 4
        for (uint32_t i = 0; i < a.groups; ++i) {
            const S o = best_of[i];
            const bool close = sizeof(S) == 4 && i != sub && o != mine && o > masked && mine > masked &&
                               fabs(o - mine) <= off + rel * (size + best_of[a.groups + i]);
            // equal scores are a tie if they are exact, or if nothing is left in both
            const bool tie = i != sub && o == mine && (off == S(0) || mine == masked);
            near += close || (i != sub && o == mine && !tie);
            before += (o > mine && !close) || (tie && i < sub);
        }
        kept = before < a.top_groups;
        open = kept && before + near >= a.top_groups;
    }
    const uint32_t shift = lane - sub;
    const uint64_t mask = L == kWave ? ~0ull : (1ull << (L & 63)) - 1;
    *unclear = ((ballot(open) >> shift) & mask) != 0;
    return (ballot(kept) >> shift) & mask;
}

template <int ELEM, int L, int V>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_kernel(RouteArgs a) {
    using T = typename Elem<ELEM>::T;
    constexpr uint32_t R = kWave / L;   // rows of a wave
    __shared__ Candidate s_list[kRouteWaves * R][L];
    extern __shared__ double s_groups[];   // with groups: a row's scores, then its groups' (as f32 in the same place)
    const uint32_t lane = threadIdx.x & (kWave - 1);
    const uint32_t sub = lane & (L - 1);
    const uint32_t slot = threadIdx.x / L;   // the row's place in the block
    const uint32_t row_or_more = block_id() * (kRouteWaves * R) + slot;
    const bool active = row_or_more < a.rows;
    const uint32_t row = active ? row_or_more : a.rows - 1;   // every lane takes part in the exchanges
    const T* in = static_cast<const T*>(a.scores) + row * a.row_stride;
    const uint32_t first = sub * V;
    const uint32_t real = first < a.experts ? a.experts - first : 0u;   // of the lane's V, those that exist
    const bool biased = a.bias != nullptr;
    const bool by_p = biased || (a.groups > 1 && a.group_best == 2);   // something goes by p, not by the scores

    float x[V], bias[V];
    load_some<V>(in + (real ? first : 0u), real, -kInf, x);
    if (biased) load_some<V>(a.bias + (real ? first : 0u), real, 0.0f, bias);

    // p in f32, in key[]; the softmax's sum in 64 bits
    Prob prob{a.sigmoid, false, 0.0, 1.0};
    float key[V];
    if (!a.sigmoid) {
        float m = x[0];
        bool nan = x[0] != x[0];
#pragma unroll
        for (int j = 1; j < V; ++j) {
            m = fmaxf(m, x[j]);
            nan |= x[j] != x[j];
        }
        m = lanes_max<L>(m);
        const uint64_t nans = ballot(nan) >> (lane - sub);
        prob.m = m != m ? -__builtin_huge_val() : static_cast<double>(m);
        prob.nan = (L == kWave ? nans : nans & ((1ull << (L & 63)) - 1)) != 0;
        if (by_p || !a.renormalize) {   // otherwise the sum cancels
            double sum = 0.0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const double e = exp64(static_cast<double>(x[j]) - prob.m);   // behind the last expert 0
                key[j] = static_cast<float>(e);
                sum += e;
                if (j & 1) __builtin_amdgcn_sched_barrier(0);   // all at once would take every register
            }
            prob.sum = lanes_sum<L>(sum);
            const float inv = prob.nan || m == kInf ? __builtin_nanf("") : static_cast<float>(1.0 / prob.sum);
#pragma unroll
            for (int j = 0; j < V; ++j) key[j] *= inv;
        }
    } else if (by_p) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            key[j] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[j] * -1.44269504088896341f));
    }

    // What the groups go by (by[]), and what the experts go by (key[])
    float by[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (biased) key[j] += bias[j];
        by[j] = by_p ? key[j] : x[j];
        const bool masked = !(x[j] > -kInf);
        if (masked || !(by[j] > -kInf)) by[j] = -kInf;
        key[j] = static_cast<uint32_t>(j) >= real ? __builtin_nanf("") : biased ? by[j] : masked ? -kInf : x[j];
    }
    // The same s in 64 bits
    auto exact = [&](float v, uint32_t e, bool masked) {
        if (masked) return kMasked;
        return biased ? prob(v) + static_cast<double>(a.bias[e]) : static_cast<double>(v);
    };

    if (a.groups > 1) {
        const uint32_t size = a.experts / a.groups;
        float* score = reinterpret_cast<float*>(s_groups + slot * (a.experts + a.groups));
        const uint32_t p = size / V;
        if (p * V == size && (p & (p - 1)) == 0) {   // whole lanes to a group, a power of two of them
            float most = by[0], next = -kInf;
#pragma unroll
            for (int j = 1; j < V; ++j) {
                next = fmaxf(next, fminf(most, by[j]));
                most = fmaxf(most, by[j]);
            }
            group_score(a, most, next, sub, p, -kInf, score + a.experts);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (static_cast<uint32_t>(j) < real) score[first + j] = by[j];
            wave_fence();
            group_scores<L>(a, score, score + a.experts, -kInf);
        }
        bool unclear;
        uint64_t kept = kept_groups<L, float>(a, score + a.experts, -kInf, by_p ? 4 * kOff : 0.0f,
                                              by_p ? 2 * kOffRel : 0.0f, &unclear);
        if (ballot(unclear) != 0) {
            double* wide = s_groups + slot * (a.experts + a.groups);
            wave_fence();
#pragma unroll 1
            for (uint32_t j = 0; j < V; ++j) {
                const uint32_t e = first + j;
                if (j < real) {
                    const float v = static_cast<float>(in[e]);
                    const double p = by_p ? prob(v) + (biased ? static_cast<double>(a.bias[e]) : 0.0) : v;
                    wide[e] = v > -kInf && p > -__builtin_huge_val() ? p : kMasked;
                }
            }
            wave_fence();
            bool none;
            group_scores<L>(a, wide, wide + a.experts, kMasked);
            const uint64_t sure = kept_groups<L, double>(a, wide + a.experts, kMasked, 0.0, 0.0, &none);
            kept = unclear ? sure : kept;
        }
        uint32_t g = first / size, in_group = first - g * size;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (!((kept >> (g & 63)) & 1ull)) key[j] = __builtin_nanf("");
            if (++in_group == size) {
                in_group = 0;
                ++g;
            }
        }
    }

    // A threshold that at least top_k of the row reach: the top_k-th of its lanes'
    // best.  An expert among the first top_k in 64 bits is no further below it
    // in f32 than twice what s may be off.
    float best = key[0];
#pragma unroll
    for (int j = 1; j < V; ++j) best = fmaxf(best, key[j]);
    const uint32_t sorted = lanes_sort_desc<L>(order32(best));
    const uint32_t kth = __shfl(sorted, static_cast<int>(lane - sub + (a.top_k <= L ? a.top_k - 1 : L - 1)), kWave);
    float tau = -kInf;   // fewer lanes have one that is not masked: every one is a candidate
    if (a.top_k <= L && kth > order32(-kInf)) {
        tau = value_of_order32(kth);
        if (biased && tau < kInf) tau -= 2 * (kOff + kOffRel * fabsf(tau));
    }

    // What reaches it is collected; where that is more than the list holds, the
    // choices are taken one after the other instead.
    uint32_t count = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) count += key[j] >= tau;
    const uint32_t incl = wave_inclusive_sum(count);
    const uint32_t last = __shfl(incl, static_cast<int>(lane | (L - 1)), kWave);
    const uint32_t previous = __shfl(incl, static_cast<int>((lane - sub - 1) & (kWave - 1)), kWave);   // by every lane
    const uint32_t before = lane >= L ? previous : 0u;
    const uint32_t found = last - before;
    const bool fits = found <= L;
    constexpr uint32_t kMaskedBit = 1u << 31;
    if (fits) {
        uint32_t at = incl - count - before;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (key[j] >= tau) {
                s_list[slot][at].x = x[j];
                s_list[slot][at++].e = (first + j) | (key[j] > -kInf ? 0u : kMaskedBit);
            }
    }
    wave_fence();
    // Lane i has candidate i; its place is the number of candidates before it.
    bool chosen = fits && sub < found;
    Candidate c{kExcluded, -kInf, 0u};
    if (chosen) {
        c.x = s_list[slot][sub].x;
        c.e = s_list[slot][sub].e;
        const bool masked = (c.e & kMaskedBit) != 0;
        c.e &= ~kMaskedBit;
        c.s = exact(c.x, c.e, masked);
        s_list[slot][sub] = c;
    }
    wave_fence();
    uint32_t place = 0;
    const uint32_t most = lanes_max(fits ? found : 0u);
#pragma unroll 4
    for (uint32_t i = 0; i < most; ++i) {
        const Candidate o = s_list[slot][i < found ? i : 0u];
        place += i < found && (o.s > c.s || (o.s == c.s && o.e < c.e));
    }
    chosen = chosen && place < a.top_k;
    if (ballot(!fits) != 0) {
        double s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s[j] = key[j] != key[j] ? kExcluded : exact(x[j], first + j, !(key[j] > -kInf));
            __builtin_amdgcn_sched_barrier(0);
        }
        for (uint32_t r = 0; r < a.top_k; ++r) {
            double mine = s[0];
            float v = x[0];
            uint32_t at = 0;
#pragma unroll
            for (int j = 1; j < V; ++j)
                if (s[j] > mine) {
                    mine = s[j];
                    v = x[j];
                    at = j;
                }
            const uint64_t with = ballot(mine == lanes_max<L>(mine)) >> (lane - sub);
            const uint32_t from = static_cast<uint32_t>(__builtin_ctzll(with));   // the lowest lane of the row
            const uint32_t e = __shfl(first + at, static_cast<int>(lane - sub + from), kWave);
            const float xe = __shfl(v, static_cast<int>(lane - sub + from), kWave);
            if (sub == from) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (j == static_cast<int>(at)) s[j] = kExcluded;
            }
            if (!fits && sub == r) {
                c = Candidate{0.0, xe, e};
                place = r;
                chosen = true;
            }
        }
    }

    const double p = chosen ? prob(c.x) : 0.0;
    double w = static_cast<double>(a.scale) * p;
    if (a.renormalize) {
        const double sum = lanes_sum<L>(p);
        w = sum == 0.0 ? 0.0 : w / sum;
    }
    if (chosen && active) {
        const uint64_t to = static_cast<uint64_t>(row) * a.top_k + place;
        a.ids[to] = c.e;
        a.weights[to] = static_cast<float>(w);
    }
}

constexpr size_t kGradLds = 32768;   // a block's: five fit a CU

// The gradient.  Every lane has one choice, whose term (summed over the choices
// of its expert) it puts into the row's LDS copy, which starts as zeros; then
// the row's lanes write it in 16-byte vectors next to each other, with the
// softmax's term that reaches every expert where the weights are not
// renormalised.  As many rows to a wave as top_k allows: the time of a wave is that
// of its dependent reads (32768 rows of 512 f32, renormalised softmax: 14.3 us
// at four rows a wave, 4.7 TB/s written; 23 at one).
template <int ELEM, int L, bool SPREAD>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_grad_kernel(RouteGradArgs a) {
    using T = typename Elem<ELEM>::T;
    constexpr uint32_t N = 16 / sizeof(T);
    constexpr uint32_t S = (L == kWave ? 16 : 8) / N;   // steps of a row whose scores are read, see grad_elem
    extern __shared__ float s_rows[];   // [rows of the block][experts, rounded up to whole steps]
    const uint32_t lane = threadIdx.x & (kWave - 1);
    const uint32_t sub = lane & (L - 1);
    const uint32_t slot = threadIdx.x / L;
    const uint32_t row_or_more = block_id() * (blockDim.x / L) + slot;
    const bool active = row_or_more < a.rows;
    const uint32_t row = active ? row_or_more : a.rows - 1;
    const T* in = static_cast<const T*>(a.scores) + row * a.row_stride;
    const uint32_t steps = (a.experts + L * N - 1) / (L * N);
    float* dx = s_rows + slot * (steps * L * N);

    const bool mine = sub < a.top_k;
    const uint64_t at = static_cast<uint64_t>(row) * a.top_k + (mine ? sub : 0u);
    const uint32_t id = mine ? a.ids[at] : 0xFFFFFFFFu;
    const float w = a.weights[at];
    const float dw = a.dweights[at];
    const float score = a.sigmoid && id < a.experts ? static_cast<float>(in[id]) : 0.0f;
    for (uint32_t i = sub; i < steps * (L * N); i += L) dx[i] = 0.0f;

    // SPREAD (softmax, not renormalised): every expert's exp(x - m), in registers
    float p[S][N];
    float sum = 0.0f;
    if (SPREAD) {
        float m = -__builtin_huge_valf();
#pragma unroll
        for (uint32_t i = 0; i < S; ++i) {
            const uint32_t e = (i * L + sub) * N;
            const bool real = e < a.experts;
            load_some<N>(in + (real ? e : 0u), real ? a.experts - e : 0u, -__builtin_huge_valf(), p[i]);
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) m = fmaxf(m, p[i][j]);
        }
        m = lanes_max<L>(m);
#pragma unroll
        for (uint32_t i = 0; i < S; ++i)
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) {
                p[i][j] = expf(p[i][j] - m);
                sum += (i * L + sub) * N + j < a.experts ? p[i][j] : 0.0f;
            }
        sum = lanes_sum<L>(sum);
        if (m == -__builtin_huge_valf()) sum = 0.0f;   // nothing is left: p = 0 (and d = 0, or NaN where the weights are)
    }

    const float d = lanes_sum<L>(mine ? dw * w : 0.0f);
    float part = w * (a.renormalize ? dw - d / a.scale : dw);
    if (a.sigmoid) {   // 1 - p, from the exponential that does not overflow
        const float e = expf(-fabsf(score));
        part *= (score > 0.0f ? e : 1.0f) / (1.0f + e);
    }
    float term = 0.0f;
    for (uint32_t r = 0; r < a.top_k; ++r) {
        const uint32_t e = __shfl(id, static_cast<int>(lane - sub + r), kWave);
        const float g = __shfl(part, static_cast<int>(lane - sub + r), kWave);
        term += e == id ? g : 0.0f;
    }
    wave_fence();
    if (id < a.experts) dx[id] = term;   // the same from every lane of the expert
    wave_fence();

    T* out = static_cast<T*>(a.dscores) + row * a.dscores_stride;
    auto write = [&](uint32_t i, const float* pi) {
        const uint32_t e = (i * L + sub) * N;
        if (e >= a.experts) return;
        float v[N];
#pragma unroll
        for (uint32_t j = 0; j < N; ++j) v[j] = dx[e + j];
        if (SPREAD) {
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) v[j] = fmaf(-(sum == 0.0f ? 0.0f : pi[j] / sum), d, v[j]);
        }
        if (active) store_some<N>(out + e, a.experts - e, v);
    };
    if (SPREAD) {
#pragma unroll
        for (uint32_t i = 0; i < S; ++i) write(i, p[i]);
    } else {
        for (uint32_t i = 0; i < steps; ++i) write(i, nullptr);
    }
}

template <int ELEM, int L, int V>
hipError_t route_shape(const RouteArgs& a, hipStream_t stream) {
    constexpr uint32_t rows = kRouteWaves * kWave / L;
    const size_t lds = a.groups > 1 ? rows * (a.experts + a.groups) * sizeof(double) : 0;
    timing_before(stream, RS_KERNEL_ROUTE);
    route_kernel<ELEM, L, V><<<many_blocks((a.rows + rows - 1) / rows), kRouteWaves * kWave, lds, stream>>>(a);
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

template <int ELEM, int L, bool SPREAD>
hipError_t grad_lanes(const RouteGradArgs& a, hipStream_t stream) {
    constexpr uint32_t step = L * (16 / sizeof(typename Elem<ELEM>::T));
    const size_t row_lds = (a.experts + step - 1) / step * step * sizeof(float);
    uint32_t waves = kRouteWaves;
    while (waves > 1 && waves * (kWave / L) * row_lds > kGradLds) waves /= 2;
    const uint32_t rows = waves * kWave / L;
    timing_before(stream, RS_KERNEL_ROUTE_GRAD);
    route_grad_kernel<ELEM, L, SPREAD><<<many_blocks((a.rows + rows - 1) / rows), waves * kWave, rows * row_lds, stream>>>(a);
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

template <int ELEM, int L>
hipError_t route_lanes(const RouteArgs& a, hipStream_t stream) {
    if (a.experts <= L) return route_shape<ELEM, L, 1>(a, stream);
    if (a.experts <= 2 * L) return route_shape<ELEM, L, 2>(a, stream);
    if (a.experts <= 4 * L) return route_shape<ELEM, L, 4>(a, stream);
    if constexpr (L == 16) {   // at most 128 experts, see route_elem
        return route_shape<ELEM, L, 8>(a, stream);
    } else {
        if (a.experts <= 8 * L) return route_shape<ELEM, L, 8>(a, stream);
        return route_shape<ELEM, L, 16>(a, stream);
    }
}

// Lanes of a row: enough that every group has one, that a lane has at most 16
// experts (8 of 16 lanes: 256 experts on 32 lanes take 11.8 us for 16384 rows,
// 15.8 on 16; 512 on 32 lanes 25 us for 32768 rows, 33 on 64), and that there
// are twice top_k: about 1.4 top_k of a row reach the top_k-th of the lanes'
// bests then, and the list of candidates has a place for each lane.  Experts
// are spread over all lanes for the same reason; kept groups may leave fewer
// lanes than top_k with one (one group of 64 of 512 experts is 4 lanes), and the
// row then goes the slow way.
template <int ELEM>
hipError_t route_elem(const RouteArgs& a, hipStream_t stream) {
    if (a.experts <= 128 && a.top_k <= 8 && a.groups <= 16) return route_lanes<ELEM, 16>(a, stream);
    if (a.experts <= 512 && a.top_k <= 16 && a.groups <= 32) return route_lanes<ELEM, 32>(a, stream);
    return route_lanes<ELEM, 64>(a, stream);
}

// A lane for each choice; and where the scores are read, lanes enough that a
// lane's registers hold its share: 8 elements of 16 or 32 lanes, 16 of 64.
template <int ELEM>
hipError_t grad_elem(const RouteGradArgs& a, hipStream_t stream) {
    if (!a.sigmoid && !a.renormalize) {
        if (a.top_k <= 16 && a.experts <= 128) return grad_lanes<ELEM, 16, true>(a, stream);
        if (a.top_k <= 32 && a.experts <= 256) return grad_lanes<ELEM, 32, true>(a, stream);
        return grad_lanes<ELEM, 64, true>(a, stream);
    }
    if (a.top_k <= 16) return grad_lanes<ELEM, 16, false>(a, stream);
    if (a.top_k <= 32) return grad_lanes<ELEM, 32, false>(a, stream);
    return grad_lanes<ELEM, 64, false>(a, stream);
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
