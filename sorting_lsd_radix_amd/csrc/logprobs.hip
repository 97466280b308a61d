// logprobs.hip -- log probabilities of given tokens with entropy, rank and
// top alternatives, and their gradient for the logits.
//
// One read of a row gives its softmax statistics: every thread keeps a
// reference r, s = sum of 2^d and t = sum of d 2^d with d = (x - r) a,
// a = scale * log2(e), and the largest x it has seen; sums with different
// references join as s 2^delta, (t + s delta) 2^delta with delta = (r - m) a.
// Then ln of the sum of exp is c m + ln s, and the entropy ln s - ln2 t / s.
// A row is one block's work, or, where rows are few, several blocks' (parts),
// whose results a second launch joins.
//
// What bounds it: at 2048 rows of 131072 bf16 logits with 8 alternatives the
// vector units (about 10 instructions an element, exp2 among them, busy in all
// of the compute units' cycles) as much as the memory: 537 MB in 101-111 us,
// 4.8-5.3 TB/s, where a kernel that only reads the same rows takes 83; in f32
// (1.07 GB) 6.4 TB/s.  The gradient moves 1.07 GB in 172-187 us, 5.8-6.2 TB/s,
// the rate of an elementwise stream.
#include "internal.hpp"
#include "rows_common.hpp"

namespace rs {

namespace {

constexpr int kLpBlock = 256;
constexpr int kLpWaves = kLpBlock / kWave;
// Parts of a row: enough for about kLpBlocks blocks (501 rows of 32003 f32 with 8
// alternatives 19 us; aiming at 2048 blocks 23, at 4096 27: every part sorts a
// list), none smaller than kLpMinPart elements (4 rows of 131072 bf16 with 20:
// both launches 17 us; parts of 2048 16.5, of 8192 17.5).
constexpr uint32_t kLpMinPart = 4096;
constexpr uint32_t kLpMaxParts = 64;
constexpr uint32_t kLpBlocks = 1024;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kInf = __builtin_huge_valf();
// A sum's reference moves when the largest x is further than this from it, in
// powers of two: far below f32's range (sums reach 2^30 * 2^16), and near
// enough that the rounding of d (16 * 2^-24) stays under a millionth.  That is
// the price of one fused multiply-add for d: a difference from the row's own
// largest would be off by the rounding of its own size only.
constexpr float kMaxShift = 16.0f;
// Largest |r a|: c = -r a is off by up to 2^-24 of it, which has to stay a small
// shift of the reference (an eighth).  Where a part's largest |x a| is over
// kMaxLargest (logits of some 7e5 at scale 1, or the lowest value of a type that
// masks a whole row), its sums are taken again with x - m formed first; below
// that, what a thread past kMaxReference would add is below 2^-(2^20).
constexpr float kMaxReference = 0x1p21f;
constexpr float kMaxLargest = 0x1p20f;

// Where a row's parts begin and end: multiples of 8 elements, so that no
// 16-byte vector of the row is in two parts.
struct Parts {
    uint32_t count, size;
};

Parts lp_parts(uint64_t rows, uint32_t vocab) {
    uint64_t want = rows ? kLpBlocks / rows : 1;
    const uint64_t most = vocab / kLpMinPart;
    if (want > most) want = most;
    if (want > kLpMaxParts) want = kLpMaxParts;
    if (want < 1) want = 1;
    const uint32_t size = static_cast<uint32_t>(((vocab + want - 1) / want + 7) / 8 * 8);
    return Parts{(vocab + size - 1) / size, size};
}

// What is known of a set of logits: the largest, sums relative to it, and how
// many come before the target.
struct Sums {
    float m, s, t;
    uint32_t ahead;
};

__device__ __forceinline__ Sums join(const Sums& x, const Sums& y, float a) {
    Sums r;
    r.m = fmaxf(x.m, y.m);
    r.ahead = x.ahead + y.ahead;
    r.s = 0.0f;
    r.t = 0.0f;
    auto add = [&](const Sums& p) {
        if (p.s != 0.0f) {   // of nothing but -inf: adds nothing, and has no reference
            const float d = fmaxf((p.m - r.m) * a, -1000.0f);
            const float f = __builtin_amdgcn_exp2f(d);
            r.s += p.s * f;
            r.t += (p.t + p.s * d) * f;
        }
    };
    add(x);
    add(y);
    return r;
}

template <class T>
struct RowVec {
    static constexpr int N = 16 / sizeof(T);
    T v[N];
};

// STREAM: the data is read once and is not kept in the caches.
template <bool STREAM, class T>
__device__ __forceinline__ RowVec<T> load_raw(const T* at) {
    using V = AnyVec<16>::V;
    const V* p = reinterpret_cast<const V*>(at);
    V v;
    if constexpr (STREAM) v = __builtin_nontemporal_load(p);
    else v = *p;
    return __builtin_bit_cast(RowVec<T>, v);
}

// Elements v * N .. of a row of n elements; behind its end -inf.
template <class T>
__device__ __forceinline__ void load_vec(const T* in, uint32_t v, uint32_t n, float (&x)[RowVec<T>::N]) {
    constexpr uint32_t N = RowVec<T>::N;
    const uint32_t at = v * N;
    if (at + N <= n) {
        const RowVec<T> r = load_raw<false>(in + at);
#pragma unroll
        for (uint32_t j = 0; j < N; ++j) x[j] = static_cast<float>(r.v[j]);
    } else {
#pragma unroll
        for (uint32_t j = 0; j < N; ++j) x[j] = at + j < n ? static_cast<float>(in[at + j]) : -kInf;
    }
}

// A logit in a list: its order pattern, then the lower index first.  Lists
// hold 0 where they have no element.
__device__ __forceinline__ uint64_t list_key(uint32_t order, uint32_t index) {
    return (static_cast<uint64_t>(order) << 32) | static_cast<uint32_t>(~index);
}

constexpr uint32_t kLpCandidates = 512;   // logits that a block's threshold may let through

struct SelectShared {
    uint64_t cand[kLpCandidates];
    uint32_t max[kLpWaves][kWave];
    uint32_t flagged[kLpBlock];
    uint32_t flags, count, tau;
    uint32_t bins[256];
    uint32_t wave[2][kLpWaves];
    uint32_t digit, need, found;
    uint64_t top[kWave];
};

// The first `need` of a part's elements with a pattern, in index order, into
// s.top[at ..]; fewer if the part has fewer.  Returns how many (everywhere).
template <class T>
__device__ uint32_t first_of_pattern(const T* in, uint32_t n, uint32_t base, uint32_t pattern, uint32_t need, uint32_t at,
                                     SelectShared& s) {
    constexpr uint32_t N = RowVec<T>::N;
    const uint32_t tid = threadIdx.x, wave = tid / kWave, lane = tid & (kWave - 1);
    const uint32_t vecs = (n + N - 1) / N;
    uint32_t taken = 0;
    for (uint32_t v0 = 0, it = 0; v0 < vecs && taken < need; v0 += kLpBlock, ++it) {
        const uint32_t v = v0 + tid;
        uint32_t mine = 0;
        if (v < vecs) {
            float x[N];
            load_vec(in, v, n, x);
            for (uint32_t j = 0; j < N; ++j)
                if (v * N + j < n && order32(x[j]) == pattern) mine |= 1u << j;
        }
        const uint32_t own = __popc(mine);
        const uint32_t incl = wave_inclusive_sum(own);
        if (lane == kWave - 1) s.wave[it & 1][wave] = incl;
        __syncthreads();
        uint32_t rank = taken + incl - own;
        for (uint32_t w = 0; w < kLpWaves; ++w) {
            const uint32_t c = s.wave[it & 1][w];
            if (w < wave) rank += c;
            taken += c;
        }
        for (uint32_t j = 0; j < N; ++j)
            if ((mine >> j) & 1u) {
                if (rank < need) s.top[at + rank] = list_key(pattern, base + v * N + j);
                ++rank;
            }
    }
    __syncthreads();
    return taken < need ? taken : need;
}

// The first k (at most n) of a row part's n elements in the row's order,
// whatever they are, by a radix select on the order patterns: four counts of
// 8-bit digits find the k-th pattern, then the patterns above it are
// collected, and of those equal to it the first by index.  s.top[0, k)
// receives the keys, in any order.
template <class T>
__device__ void radix_select(const T* in, uint32_t n, uint32_t base, uint32_t k, SelectShared& s) {
    constexpr uint32_t N = RowVec<T>::N;
    const uint32_t tid = threadIdx.x, wave = tid / kWave, lane = tid & (kWave - 1);
    const uint32_t vecs = (n + N - 1) / N;
    uint32_t prefix = 0, need = k;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) s.bins[tid] = 0;
        __syncthreads();
        for (uint32_t v = tid; v < vecs; v += kLpBlock) {
            float x[N];
            load_vec(in, v, n, x);
            for (uint32_t j = 0; j < N; ++j) {
                const uint32_t o = order32(x[j]);
                const uint32_t digit = (o >> shift) & 255u;
                const bool counts = v * N + j < n && (shift == 24 || ((o ^ prefix) >> (shift + 8)) == 0);
                // ties bring rows here: lanes with one digit count it together
                const uint64_t all = ballot(counts);
                if (all == 0) continue;
                const uint32_t leader = static_cast<uint32_t>(__builtin_ctzll(all));
                const uint32_t theirs = __shfl(digit, static_cast<int>(leader), kWave);
                if (ballot(counts && digit == theirs) == all) {
                    if (lane == leader) atomicAdd(&s.bins[digit], static_cast<uint32_t>(__builtin_popcountll(all)));
                } else if (counts) {
                    atomicAdd(&s.bins[digit], 1u);
                }
            }
        }
        __syncthreads();
        // thread t holds digit 255 - t: how many have a larger digit
        const uint32_t own = tid < 256 ? s.bins[255 - tid] : 0u;
        const uint32_t incl = wave_inclusive_sum(own);
        if (lane == kWave - 1) s.wave[0][wave] = incl;
        __syncthreads();
        uint32_t above = incl - own;
        for (uint32_t w = 0; w < wave; ++w) above += s.wave[0][w];
        if (above < need && need <= above + own) {
            s.digit = 255 - tid;
            s.need = need - above;
        }
        __syncthreads();
        prefix |= s.digit << shift;
        need = s.need;
    }
    if (tid == 0) s.found = 0;
    __syncthreads();
    if (need < k) {
        for (uint32_t v = tid; v < vecs; v += kLpBlock) {
            float x[N];
            load_vec(in, v, n, x);
            for (uint32_t j = 0; j < N; ++j) {
                const uint32_t o = order32(x[j]);
                if (v * N + j < n && o > prefix) s.top[atomicAdd(&s.found, 1u)] = list_key(o, base + v * N + j);
            }
        }
    }
    first_of_pattern(in, n, base, prefix, need, k - need, s);
}

// Writes a row's results.  Called by one wave; lane i has the i-th list key.
__device__ __forceinline__ void finish_row(const LogprobsArgs& p, uint32_t row, Sums z, float x_target,
                                           bool has_target, uint64_t key) {
    const uint32_t lane = lane_id();
    const bool empty = z.m == -kInf && z.s == 0.0f;
    if (z.m == kInf) z.s = __builtin_nanf("");
    const float ln_s = empty ? 0.0f : logf(z.s);
    auto ln_p = [&](float x) { return x == -kInf && z.s == z.s ? -kInf : (x - z.m) * p.scale - ln_s; };
    if (lane == 0) {
        p.stats[2ull * row] = z.m;
        p.stats[2ull * row + 1] = z.s;
        if (p.lse) p.lse[row] = empty ? -kInf : z.m * p.scale + ln_s;
        if (p.entropy) p.entropy[row] = empty ? 0.0f : ln_s - kLn2 * (z.t / z.s);   // s >= 1, t <= 0
        if (p.logprob) p.logprob[row] = has_target ? ln_p(x_target) : 0.0f;
        if (p.rank) p.rank[row] = has_target && x_target == x_target ? z.ahead : 0xFFFFFFFFu;
    }
    if (lane < p.top_k) {
        const float x = value_of_order32(static_cast<uint32_t>(key >> 32));
        p.top_ids[static_cast<uint64_t>(row) * p.top_k + lane] = ~static_cast<uint32_t>(key);
        p.top_logprobs[static_cast<uint64_t>(row) * p.top_k + lane] = ln_p(x);
    }
}

// A thread's running sums over d = x a + c, in powers of two: c = -r a puts the
// reference r at 0.  One fused multiply-add gives d, rounded once, and every
// use of the reference goes through the same c, so that its rounding cancels.
struct Running {
    float m = -kInf, c = 0.0f, s = 0.0f, t = 0.0f;

    // x - y of the two rounded numbers.  Where the compiler fuses a product into it, the sums so far
    // are moved by the product before its rounding, which is off by up to 2^-24 |m a| from
    // where the terms to come are counted from: with logits around -7e5 s was off by a part in 150.
    static __device__ __forceinline__ float difference(float x, float y) {
#pragma clang fp contract(off)
        return x - y;
    }

    // Called with a new largest m: moves the reference there, unless it is near
    // enough, or too large for c (slow_sums then).
    __device__ __forceinline__ void reference(float a) {
        if (!(fabsf(fmaf(m, a, c)) <= kMaxShift) && fabsf(m * a) <= kMaxReference) {
            const float to = -m * a;
            const float d = fmaxf(difference(to, c), -1000.0f);
            const float f = __builtin_amdgcn_exp2f(d);
            if (s != 0.0f) {
                t = (t + s * d) * f;
                s *= f;
            }
            c = to;
        }
    }

    // Adds the logits of one step; `top` is the largest of them.
    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N], float top, float a) {
        m = fmaxf(m, top);
        reference(a);
        float s2[2] = {0.0f, 0.0f}, t2[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float d = fmaf(x[j], a, c);
            const float e = __builtin_amdgcn_exp2f(d);
            s2[j & 1] += e;
            t2[j & 1] = fmaf(e, fmaxf(d, -1000.0f), t2[j & 1]);   // a masked logit adds 0 * -1000
        }
        s += s2[0] + s2[1];
        t += t2[0] + t2[1];
    }

    // The sums with the largest logit as the reference.  Its own term is 1 and adds nothing to t:
    // what add() took for it is taken out of the sums before they are scaled, so that s is never
    // below 1 (no probability above 1) and a row with one token left gives s = 1 and t = 0.
    __device__ __forceinline__ Sums relative_to_largest(float a) const {
        if (!(fabsf(m * a) <= kMaxReference)) return Sums{m, s == s ? 0.0f : s, 0.0f, 0u};
        const float d = fmaf(m, a, c);
        const float f = __builtin_amdgcn_exp2f(-d);
        const float e = __builtin_amdgcn_exp2f(d);
        const float rest = s - e;
        if (rest <= 0.0f) return Sums{m, 1.0f, 0.0f, 0u};   // nothing else, or less than s's roundings
        const float moved = (t - e * d - rest * d) * f;      // no term of t is above 0
        return Sums{m, 1.0f + rest * f, moved < 0.0f ? moved : 0.0f, 0u};
    }
};

// Where |largest * a| > kMaxLargest: the block's sums again, with x - m formed
// before the product.  m is finite.
template <class T>
__device__ __attribute__((noinline)) Sums slow_sums(const T* in, uint32_t n, float m, float a, Sums* s_sums) {
    constexpr uint32_t N = RowVec<T>::N;
    const uint32_t tid = threadIdx.x;
    float s = 0.0f, t = 0.0f;
    for (uint32_t v = tid; v < (n + N - 1) / N; v += kLpBlock) {
        float x[N];
        load_vec(in, v, n, x);
        for (uint32_t j = 0; j < N; ++j) {
            const float d = (x[j] - m) * a;
            const float e = __builtin_amdgcn_exp2f(d);
            s += e;
            t = fmaf(e, fmaxf(d, -1000.0f), t);
        }
    }
    s = lanes_sum(s);
    t = lanes_sum(t);
    __syncthreads();
    if ((tid & (kWave - 1)) == 0) s_sums[tid / kWave] = Sums{m, s, t, 0u};
    __syncthreads();
    Sums z{m, 0.0f, 0.0f, 0u};
    for (uint32_t w = 0; w < kLpWaves; ++w) {
        z.s += s_sums[w].s;
        z.t += s_sums[w].t;
    }
    return z;
}

// Logits before the target by comparisons of single elements, where the
// target's logit is -inf (no value is below it, see the kernel).
template <class T>
__device__ __attribute__((noinline)) uint32_t slow_ahead(const T* in, uint32_t n, uint32_t base, uint32_t target) {
    constexpr uint32_t N = RowVec<T>::N;
    uint32_t ahead = 0;
    for (uint32_t v = threadIdx.x; v < (n + N - 1) / N; v += kLpBlock) {
        float x[N];
        load_vec(in, v, n, x);
        for (uint32_t j = 0; j < N; ++j)
            ahead += x[j] > -kInf || (x[j] == -kInf && base + v * N + j < target);
    }
    return lanes_sum(ahead);
}

// The steps in which a thread read its share of a part: 16 elements each (U
// vectors, U * kLpBlock vectors apart from step to step), then single vectors.
// Of them TOP keeps the largest steps' largest logits, and the first's number.
struct Steps {
    float best = -kInf, next = -kInf;   // the two largest of the steps' largest logits
    uint32_t at = 0;                    // the step of `best`
    __device__ __forceinline__ void add(float top, uint32_t step) {
        at = top > best ? step : at;
        next = __builtin_amdgcn_fmed3f(top, best, next);
        best = fmaxf(best, top);
    }
};

// The first k <= n of a part's logits: wave 0 returns them, lane i the i-th.
//
// The k-th largest of the threads' largest logits is a threshold that at
// least k logits reach, and in a row without many ties hardly more: only the
// threads whose largest reaches it can hold one of the first k.  Such a thread
// reads the step that holds its largest again; where a second step of it
// reaches the threshold too, a whole wave reads the thread's share.  (Reading
// whole shares in every case cost 20 us of 123 at 2048 rows of 131072 bf16
// logits.)  What reaches the threshold is collected and sorted by (value,
// index).  Where more is collected than the list takes, ties as a rule, only
// what is above the threshold is collected, and the first ties by index follow
// (where masks leave fewer than k, the first masked ones); where that is too much
// too (the best logits crowded in few shares), the radix select reads the part.
template <class T>
__device__ __forceinline__ uint64_t best_of_part(const T* in, uint32_t n, uint32_t base, uint32_t k,
                                                 const Steps& steps, uint32_t full_steps, SelectShared& s) {
    constexpr uint32_t N = RowVec<T>::N;
    constexpr uint32_t U = 16 / N;
    const uint32_t tid = threadIdx.x, wave = tid / kWave, lane = tid & (kWave - 1);
    const uint32_t vecs = (n + N - 1) / N;
    const bool all = n <= kLpCandidates;   // no threshold: everything is collected
    const uint32_t lowest = order32(-kInf);
    uint32_t tau = 0;
    auto collect = [&](uint32_t v) {
        float x[N];
        load_vec(in, v, n, x);
#pragma unroll
        for (uint32_t j = 0; j < N; ++j) {
            const uint32_t o = order32(x[j]);
            if (o >= tau && v * N + j < n) {
                const uint32_t at = atomicAdd(&s.count, 1u);
                if (at < kLpCandidates) s.cand[at] = list_key(o, base + v * N + j);
            }
        }
    };
    if (tid == 0) s.flags = s.count = 0;
    if (all) {
        __syncthreads();
        for (uint32_t v = tid; v < vecs; v += kLpBlock) collect(v);
    } else {
        // of 64 groups of four threads' bests while top_k is at most half of
        // them (one sort in every wave), of all threads' above
        const uint32_t mine = order32(steps.best);
        uint32_t kth;
        if (k <= kWave / 2) {
            const uint32_t of_four = lanes_max<4>(mine);
            if ((lane & 3) == 0) s.max[0][wave * (kWave / 4) + lane / 4] = of_four;
            __syncthreads();
            kth = __shfl(wave_sort_desc(s.max[0][lane]), static_cast<int>(k - 1), kWave);
        } else {
            uint32_t list = wave_sort_desc(mine);
#pragma unroll
            for (uint32_t half = kLpWaves / 2; half > 0; half >>= 1) {
                if (wave >= half && wave < 2 * half) s.max[wave][lane] = list;
                __syncthreads();
                if (wave < half) list = wave_merge_desc(list, s.max[wave + half][lane]);
            }
            if (wave == 0 && lane == k - 1) s.tau = list;
            __syncthreads();
            kth = s.tau;
        }
        tau = kth > lowest ? kth : lowest + 1;   // never the masked ones
        for (int attempt = 0;; ++attempt) {
            if (mine >= tau) {
                if (order32(steps.next) >= tau) {
                    s.flagged[atomicAdd(&s.flags, 1u)] = tid;
                } else {
                    const bool whole = steps.at < full_steps;
                    const uint32_t v = tid + kLpBlock * (whole ? steps.at * U : full_steps * U + steps.at - full_steps);
                    for (uint32_t u = 0; u < (whole ? U : 1); ++u) collect(v + u * kLpBlock);
                }
            }
            __syncthreads();
            for (uint32_t i = wave; i < s.flags; i += kLpWaves) {
                if (__hip_atomic_load(&s.count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) > kLpCandidates) break;
                for (uint32_t v = s.flagged[i] + lane * kLpBlock; v < vecs; v += kWave * kLpBlock) collect(v);
            }
            __syncthreads();
            if (s.count <= kLpCandidates || attempt == 1) break;
            __syncthreads();   // too many reach the threshold: mostly ties, so only what is above it
            if (tid == 0) s.flags = s.count = 0;
            ++tau;
            __syncthreads();
        }
    }
    __syncthreads();
    const uint32_t count = s.count;
    if (count > kLpCandidates || count < k) {
        // fewer than k reach the threshold where it was raised over ties, or stood
        // above the masked ones: those, and then the first of the ties or masked
        // ones (unless NaN has to fill up too)
        const bool few = count < k && first_of_pattern(in, n, base, tau - 1, k - count, count, s) == k - count;
        if (!few) radix_select(in, n, base, k, s);
        if (few && tid < count) s.top[tid] = s.cand[tid];
        wave_fence();   // count < k: wave 0 wrote them
        return wave == 0 ? wave_sort_desc(lane < k ? s.top[lane] : uint64_t{0}) : 0;
    }
    uint64_t key = 0;
    if (wave == 0 && count <= kWave) {
        // each lane's candidate goes to the place of as many as are before it
        const uint64_t own = lane < count ? s.cand[lane] : uint64_t{0};
        uint32_t place = 0;
#pragma unroll 8
        for (uint32_t i = 0; i < count; ++i) place += s.cand[i] > own;
        if (lane < count) s.top[place] = own;
        wave_fence();
        key = lane < count ? s.top[lane] : uint64_t{0};
    } else if (wave == 0) {
        for (uint32_t i = 0; i < count; i += kWave) {
            const uint64_t next = wave_sort_desc(i + lane < count ? s.cand[i + lane] : uint64_t{0});
            key = i == 0 ? next : wave_merge_desc(key, next);
        }
    }
    return key;
}

// Block (part, row): the sums and, with top_k, the list of one part of a row.
// With one part the row is finished here; otherwise part q of a row leaves
// its sums at sums[row * parts + q] and its list at lists[(row * parts + q) * top_k].
//
// Thread t reads the 16-byte vectors t, t + 256, ... of the part, 16 elements
// a step, the next step's loads in flight.  Logits before the target are
// counted as wave masks (a compare and scalar instructions): behind the
// target those above it, in front of it those above the next value below it,
// which are the ones not below it; the vector that holds the target is
// counted as behind it and its equal logits in front of it added.
template <int ELEM, bool TOP, bool STREAM>
__global__ __launch_bounds__(kLpBlock) void logprobs_kernel(LogprobsArgs p, Parts parts, Sums* __restrict__ sums,
                                                            uint64_t* __restrict__ lists) {
    using T = typename Elem<ELEM>::T;
    constexpr uint32_t N = RowVec<T>::N;
    constexpr uint32_t U = 16 / N;   // vectors of a step
    __shared__ Sums s_sums[kLpWaves];
    __shared__ SelectShared s_select;
    const uint32_t tid = threadIdx.x, wave = tid / kWave, lane = tid & (kWave - 1);
    const uint32_t block = block_id();
    const uint32_t row = block / parts.count;
    const uint32_t part = block - row * parts.count;
    if (row >= p.rows) return;
    const uint32_t base = part * parts.size;
    const uint32_t n = p.vocab - base < parts.size ? p.vocab - base : parts.size;
    const T* whole = static_cast<const T*>(p.logits) + row * p.row_stride;
    const T* in = whole + base;
    const float a = p.scale * kLog2e;

    const uint32_t target = p.targets ? p.targets[row] : 0xFFFFFFFFu;
    const bool has_target = target < p.vocab;
    const bool rank = has_target && p.rank != nullptr;
    const float x_target = has_target ? static_cast<float>(whole[target]) : 0.0f;
    // what a counted logit is above: behind the target its logit, in front of it (vectors before
    // at_target) the next value below; +inf counts nothing
    const uint32_t xt = __float_as_uint(x_target);
    const float over_behind = rank ? x_target : kInf;
    const float over_front = !rank ? kInf
                             : (xt << 1) == 0 ? __uint_as_float(0x80000001u)
                                              : __uint_as_float((xt >> 31) ? xt + 1 : xt - 1);
    const uint32_t at_target = rank && target >= base ? (target - base) / N : 0u;

    Running r;
    Steps top_steps;
    uint32_t ahead = 0;   // of the wave
    auto count_ahead = [&](const float* x, uint32_t v) {
        const float over = v < at_target ? over_front : over_behind;
#pragma unroll
        for (uint32_t j = 0; j < N; ++j) ahead += static_cast<uint32_t>(__builtin_popcountll(ballot(x[j] > over)));
    };
    const uint32_t vecs = (n + N - 1) / N;
    const uint32_t steps = n / (kLpBlock * 16);
    if (steps > 0) {
        RowVec<T> raw[U];
        float x[16];
        auto load = [&](uint32_t i) {
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) raw[u] = load_raw<STREAM>(in + ((i * U + u) * kLpBlock + tid) * N);
        };
        auto convert = [&] {
#pragma unroll
            for (uint32_t u = 0; u < U; ++u)
#pragma unroll
                for (uint32_t j = 0; j < N; ++j) x[u * N + j] = static_cast<float>(raw[u].v[j]);
        };
        auto add = [&](uint32_t i) {
            float top = x[0];
#pragma unroll
            for (int j = 1; j < 16; ++j) top = fmaxf(top, x[j]);
            r.add(x, top, a);
            if (TOP) top_steps.add(top, i);
            if (ballot(top > over_front) != 0) {   // a likely target has few above it
#pragma unroll
                for (uint32_t u = 0; u < U; ++u) count_ahead(x + u * N, (i * U + u) * kLpBlock + tid);
            }
        };
        load(0);
        for (uint32_t i = 0; i + 1 < steps; ++i) {
            convert();
            load(i + 1);
            add(i);
        }
        convert();
        add(steps - 1);
    }
    for (uint32_t v = steps * (U * kLpBlock) + tid, i = steps; v - tid < vecs; v += kLpBlock, ++i) {   // uniform
        float x[N];
        load_vec(in, v, n, x);
        float top = x[0];
#pragma unroll
        for (uint32_t j = 1; j < N; ++j) top = fmaxf(top, x[j]);
        r.add(x, top, a);
        if (TOP) top_steps.add(top, i);
        if (ballot(top > over_front) != 0) count_ahead(x, v);
    }
    if (rank && x_target == -kInf) {
        ahead = slow_ahead(in, n, base, target);
    } else if (rank && target >= base && target - base < n && wave == 0) {
        const uint32_t at = at_target * N + lane;
        ahead += static_cast<uint32_t>(__builtin_popcountll(
            ballot(lane < N && base + at < target && static_cast<float>(in[at < n ? at : 0]) == x_target)));
    }
    Sums z = r.relative_to_largest(a);
    z = lanes_reduce(z, [&](const Sums& x, const Sums& y) { return join(x, y, a); });
    z.ahead = ahead;
    if (lane == 0) s_sums[wave] = z;
    __syncthreads();
    z = s_sums[0];
    for (uint32_t w = 1; w < kLpWaves; ++w) z = join(z, s_sums[w], a);
    if (fabsf(z.m) < kInf && fabsf(z.m * a) > kMaxLargest) {
        const uint32_t counted = z.ahead;
        z = slow_sums(in, n, z.m, a, s_sums);
        z.ahead = counted;
    }
    uint64_t key = 0;
    if (TOP) key = best_of_part(in, n, base, p.top_k < n ? p.top_k : n, top_steps, steps, s_select);
    if (wave != 0) return;
    if (parts.count == 1) {
        finish_row(p, row, z, x_target, has_target, key);
    } else {
        if (lane == 0) sums[block] = z;
        if (TOP && lane < p.top_k) lists[static_cast<uint64_t>(block) * p.top_k + lane] = key;
    }
}

// One block a row joins its parts: wave w merges the lists w, w + 8, ..., then
// the waves' lists merge in pairs.
constexpr int kLpJoinWaves = 8;
template <int ELEM>
__global__ __launch_bounds__(kLpJoinWaves* kWave) void logprobs_join_kernel(LogprobsArgs p, Parts parts,
                                                                            const Sums* __restrict__ sums,
                                                                            const uint64_t* __restrict__ lists) {
    using T = typename Elem<ELEM>::T;
    __shared__ uint64_t s_list[kLpJoinWaves][kWave];
    const uint32_t row = block_id(), wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    if (row >= p.rows) return;
    const float a = p.scale * kLog2e;
    const uint64_t first = static_cast<uint64_t>(row) * parts.count;
    Sums z{-kInf, 0.0f, 0.0f, 0u};
    uint32_t target = 0xFFFFFFFFu;
    float x_target = 0.0f;
    if (wave == 0) {
        if (lane < parts.count) z = sums[first + lane];   // at most kWave parts
        if (p.targets) target = p.targets[row];
        if (target < p.vocab)
            x_target = static_cast<float>(static_cast<const T*>(p.logits)[row * p.row_stride + target]);
    }
    uint64_t key = 0;
    if (p.top_k) {
        for (uint32_t q = wave; q < parts.count; q += kLpJoinWaves) {
            const uint64_t next = lane < p.top_k ? lists[(first + q) * p.top_k + lane] : uint64_t{0};
            key = q == wave ? next : wave_merge_desc(key, next);
        }
#pragma unroll
        for (uint32_t half = kLpJoinWaves / 2; half > 0; half >>= 1) {
            if (wave >= half && wave < 2 * half) s_list[wave][lane] = key;
            __syncthreads();
            if (wave < half) key = wave_merge_desc(key, s_list[wave + half][lane]);
        }
    }
    if (wave != 0) return;
    z = lanes_reduce(z, [&](const Sums& x, const Sums& y) { return join(x, y, a); });
    finish_row(p, row, z, x_target, target < p.vocab, key);
}
static_assert(kLpBlock == 4 * kWave, "a threshold of 64 groups of four threads");
static_assert(kLpMaxParts <= kWave, "the joining wave has a lane for each part");

// Block (part of a row, row): dx = e (c0 + c1 d) with e = 2^d, d = (x - m) a, plus
// the target's own term; the row's statistics and gradients are folded into c0
// and c1 once a thread.  Bound by the memory (figures at the top): loads around
// the caches take the same 184-187 us, stores around them 195.
constexpr uint32_t kLpGradVecs = 4;   // 16-byte vectors of a thread
template <int ELEM>
__global__ __launch_bounds__(kLpBlock) void logprobs_grad_kernel(LogprobsGradArgs p, uint32_t blocks_a_row) {
    using T = typename Elem<ELEM>::T;
    constexpr uint32_t N = RowVec<T>::N;
    const uint32_t block = block_id();
    const uint32_t row = block / blocks_a_row;
    if (row >= p.rows) return;
    const uint32_t v0 = (block - row * blocks_a_row) * (kLpBlock * kLpGradVecs) + threadIdx.x;
    const T* in = static_cast<const T*>(p.logits) + row * p.row_stride;
    T* out = static_cast<T*>(p.dlogits) + row * p.dlogits_stride;
    const float a = p.scale * kLog2e;
    const float m = p.stats[2ull * row], s = p.stats[2ull * row + 1];
    const uint32_t target = p.targets ? p.targets[row] : 0xFFFFFFFFu;
    const float g = p.dlogprob && target < p.vocab ? p.dlogprob[row] : 0.0f;
    const float h = p.dentropy ? p.dentropy[row] : 0.0f;
    const float q = p.dlse ? p.dlse[row] : 0.0f;
    const bool empty = m == -kInf && s == 0.0f;
    const float big_h = p.dentropy ? p.entropy[row] : 0.0f;
    const float c0 = empty ? 0.0f : p.scale * (q - g - (p.dentropy ? h * (big_h - logf(s)) : 0.0f)) / s;
    const float c1 = empty ? 0.0f : -p.scale * h * kLn2 / s;
    const float own = empty ? 0.0f : p.scale * g;
    const uint32_t vecs = (p.vocab + N - 1) / N;
#pragma unroll
    for (uint32_t i = 0; i < kLpGradVecs; ++i) {
        const uint32_t v = v0 + i * kLpBlock;
        if (v >= vecs) break;
        float x[N];
        load_vec(in, v, p.vocab, x);
        RowVec<T> o;
#pragma unroll
        for (uint32_t j = 0; j < N; ++j) {
            const float d = empty ? 0.0f : (x[j] - m) * a;
            const float e = __builtin_amdgcn_exp2f(d);
            float dx = e * fmaf(c1, fmaxf(d, -1000.0f), c0);
            if (v * N + j == target) dx += own;
            o.v[j] = static_cast<T>(dx);
        }
        if ((v + 1) * N <= p.vocab) {
            using V = AnyVec<16>::V;
            *reinterpret_cast<V*>(out + v * N) = __builtin_bit_cast(V, o);
        } else {
#pragma unroll
            for (uint32_t j = 0; j < N; ++j)
                if (v * N + j < p.vocab) out[v * N + j] = o.v[j];
        }
    }
}

// Above this size (the last-level cache's) logits are read around the caches:
// 2048 rows of 131072 bf16 101 -> 87 us, of f32 180 -> 157 us; below it the
// caches may still hold them (257 rows of 50021 f32: 18.6 us against 20.0).
constexpr uint64_t kLpStreamBytes = uint64_t{1} << 28;

template <int ELEM>
hipError_t logprobs_elem(const LogprobsArgs& p, void* temp, hipStream_t stream) {
    const Parts parts = lp_parts(p.rows, p.vocab);
    const uint64_t blocks = static_cast<uint64_t>(p.rows) * parts.count;
    const bool around = static_cast<uint64_t>(p.rows) * p.vocab * sizeof(typename Elem<ELEM>::T) > kLpStreamBytes;
    uint64_t* lists = static_cast<uint64_t*>(temp);
    Sums* sums = reinterpret_cast<Sums*>(lists + (parts.count > 1 ? blocks * p.top_k : 0));
    const auto kernel = p.top_k ? (around ? logprobs_kernel<ELEM, true, true> : logprobs_kernel<ELEM, true, false>)
                                : (around ? logprobs_kernel<ELEM, false, true> : logprobs_kernel<ELEM, false, false>);
    timing_before(stream, RS_KERNEL_LOGPROBS);
    kernel<<<many_blocks(blocks), kLpBlock, 0, stream>>>(p, parts, sums, lists);
    hipError_t e = hipGetLastError();
    timing_after(stream);
    if (e != hipSuccess || parts.count == 1) return e;
    timing_before(stream, RS_KERNEL_LOGPROBS_JOIN);
    logprobs_join_kernel<ELEM><<<many_blocks(p.rows), kLpJoinWaves * kWave, 0, stream>>>(p, parts, sums, lists);
    e = hipGetLastError();
    timing_after(stream);
    return e;
}

template <int ELEM>
hipError_t grad_elem(const LogprobsGradArgs& p, hipStream_t stream) {
    constexpr uint32_t kSpan = kLpBlock * kLpGradVecs * RowVec<typename Elem<ELEM>::T>::N;
    const uint32_t blocks_a_row = (p.vocab + kSpan - 1) / kSpan;
    timing_before(stream, RS_KERNEL_LOGPROBS_GRAD);
    logprobs_grad_kernel<ELEM><<<many_blocks(static_cast<uint64_t>(p.rows) * blocks_a_row), kLpBlock, 0, stream>>>(p, blocks_a_row);
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

}  // namespace

size_t logprobs_temp_bytes(uint64_t rows, uint32_t vocab, uint32_t top_k) {
    const Parts parts = lp_parts(rows, vocab);
    if (rows == 0 || parts.count == 1) return RS_NO_TEMP;
    return rows * parts.count * (sizeof(Sums) + 8 * static_cast<size_t>(top_k));
}

hipError_t launch_logprobs(int elem_type, const LogprobsArgs& p, void* temp, hipStream_t stream) {
    switch (elem_type) {
    case RS_ELEM_F32: return logprobs_elem<RS_ELEM_F32>(p, temp, stream);
    case RS_ELEM_F16: return logprobs_elem<RS_ELEM_F16>(p, temp, stream);
    default: return logprobs_elem<RS_ELEM_BF16>(p, temp, stream);
    }
}

hipError_t launch_logprobs_grad(int elem_type, const LogprobsGradArgs& p, hipStream_t stream) {
    switch (elem_type) {
    case RS_ELEM_F32: return grad_elem<RS_ELEM_F32>(p, stream);
    case RS_ELEM_F16: return grad_elem<RS_ELEM_F16>(p, stream);
    default: return grad_elem<RS_ELEM_BF16>(p, stream);
    }
}

}  // namespace rs
