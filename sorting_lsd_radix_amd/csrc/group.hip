// group.hip -- the choices of a router ordered by expert: a stable partition
// with one side for each expert.
//
// A block ranks a tile of choices: wave w holds the w-th run of 64 ITEMS
// choices in registers, 64 a row, so that (wave, row, lane) is input order.  A
// choice's rank among its expert's in the wave is the wave's count of earlier
// rows plus the peers in lower lanes, found by a ballot for each bit of the
// expert's number; sums over waves, tiles and experts give its place.  Nothing
// depends on the order in which blocks or atomics run.
//
//  * One tile: one launch does it all.
//  * Up to kShortSum counts (tiles * experts): two launches.  Every tile
//    counts its choices; then every tile sums the counts of earlier and of all
//    tiles itself, which is cheaper than a launch in between.
//  * Above: a launch in between turns the counts of each expert into the
//    tiles' offsets and a total.
//
// What bounds it: launches and dependent steps where choices are few; 131072 of
// 256 experts take 2.4 + 8.1 us (the choices and their order are 1.7 MB, but every
// block reads the 128 KB of counts), 1.3 million of 1000 experts 4.4 + 6.3 + 16 us
// (15.7 MB, the order written in scattered words).
#include "internal.hpp"
#include "device_common.hpp"

namespace rs {

namespace {

constexpr int kGroupBlock = 1024;
constexpr int kGroupWaves = kGroupBlock / kWave;
constexpr uint32_t kNone = 0xFFFFFFFFu;
// Calls in a captured graph, two launches against three: 2^14 counts 8.0 us
// against 10.9, 2^15 9.7 against 11.4, 2^16 12.7 against 11.9, 2^17 19.0 against 13.0.
constexpr uint32_t kShortSum = 1u << 15;

// Choices of a thread.  One tile up to 4096 choices: a launch less, which few
// experts gain by (2048 of 64: 5.4 us in one tile, 6.2 in two of 1024; 4096 of
// 1000: 15.7 in one, 10.0 in four).  Above, tiles of 1024, which fill the chip
// soonest (131072 of 64: 7.2 us, in tiles of 4096 9.6), and above 2^18 of 4096
// (2^20 of 256: 18.4 us, in tiles of 1024 22.6, of 16384 27; at 2^18 itself the
// two are within 1.5 us of each other, either way by the experts).
int group_items(uint64_t n) {
    if (n <= kGroupBlock) return 1;
    if (n <= 4 * kGroupBlock) return 4;
    return n <= (uint64_t{1} << 18) ? 1 : 4;
}

uint32_t group_tiles(uint64_t n) {
    const uint64_t tile = static_cast<uint64_t>(kGroupBlock) * group_items(n);
    return static_cast<uint32_t>((n + tile - 1) / tile);
}

template <int ITEMS>
__global__ __launch_bounds__(kGroupBlock) void group_count_kernel(GroupArgs a, uint32_t* __restrict__ tile_counts) {
    __shared__ uint32_t s_count[RS_MAX_EXPERTS];
    const uint32_t tid = threadIdx.x;
    const uint32_t base = blockIdx.x * (kGroupBlock * ITEMS);
    s_count[tid] = 0;
    uint32_t e[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const uint32_t i = base + j * kGroupBlock + tid;
        e[j] = i < a.n ? a.ids[i] : kNone;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j)
        if (e[j] < a.experts) atomicAdd(&s_count[e[j]], 1u);
    __syncthreads();
    if (tid < a.experts) tile_counts[static_cast<uint64_t>(blockIdx.x) * a.experts + tid] = s_count[tid];
}

// Block b, experts 16 b .. : tile_counts become the choices of earlier tiles,
// totals[e] those of all.  Thread (r, x) takes run r of 64 of the tiles for
// expert 16 b + x: sums it, then, with the sums of earlier runs, writes its
// offsets, eight loads in flight.
constexpr uint32_t kScanExperts = 16;
constexpr uint32_t kScanRuns = kGroupBlock / kScanExperts;

__global__ __launch_bounds__(kGroupBlock) void group_scan_kernel(uint32_t experts, uint32_t tiles,
                                                                 uint32_t* __restrict__ tile_counts,
                                                                 uint32_t* __restrict__ totals) {
    __shared__ uint32_t s_sum[kScanRuns][kScanExperts];
    const uint32_t r = threadIdx.x / kScanExperts, x = threadIdx.x % kScanExperts;
    const uint32_t e = blockIdx.x * kScanExperts + x;
    const bool real = e < experts;
    const uint32_t run = (tiles + kScanRuns - 1) / kScanRuns;
    const uint32_t begin = r * run < tiles ? r * run : tiles;
    const uint32_t end = begin + run < tiles ? begin + run : tiles;
    uint32_t* col = tile_counts + (real ? e : 0u);
    uint32_t c[8];
    auto load = [&](uint32_t t0) {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) c[j] = col[static_cast<uint64_t>(t0 + j < end ? t0 + j : t0) * experts];
    };
    uint32_t sum = 0;
    for (uint32_t t0 = begin; t0 < end; t0 += 8) {
        load(t0);
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) sum += t0 + j < end ? c[j] : 0u;
    }
    s_sum[r][x] = sum;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (uint32_t i = 0; i < kScanRuns; ++i) {
        const uint32_t s = s_sum[i][x];
        before += i < r ? s : 0u;
        all += s;
    }
    if (!real) return;
    if (r == 0) totals[e] = all;
    for (uint32_t t0 = begin; t0 < end; t0 += 8) {
        load(t0);
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
            if (t0 + j >= end) break;
            col[static_cast<uint64_t>(t0 + j) * experts] = before;
            before += c[j];
        }
    }
}

// Where a tile learns of the others' choices.
enum Source { kAlone, kTileCounts, kTileOffsets };

template <int ITEMS, Source SOURCE>
__global__ __launch_bounds__(kGroupBlock) void group_place_kernel(GroupArgs a, uint32_t bits,
                                                                  const uint32_t* __restrict__ tile_counts,
                                                                  const uint32_t* __restrict__ totals) {
    // [experts] words: first place of the tile's choices, first and end of the
    // padding; then [waves][experts] halves: a wave's choices, then those of
    // the tile's earlier waves
    extern __shared__ uint32_t s_base[];
    uint32_t* s_pad = s_base + a.experts;
    uint32_t* s_end = s_pad + a.experts;
    __shared__ uint32_t s_wave[kGroupWaves];
    __shared__ uint32_t s_part[2][kGroupBlock];
    __shared__ uint32_t s_length;
    const uint32_t tid = threadIdx.x, wave = tid / kWave, lane = tid & (kWave - 1);
    uint16_t* s_count = reinterpret_cast<uint16_t*>(s_end + a.experts) + wave * a.experts;   // the wave's
    const uint32_t tile = blockIdx.x;
    const uint32_t base = tile * (kGroupBlock * ITEMS) + wave * (kWave * ITEMS) + lane;

    uint32_t e[ITEMS], rank[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const uint32_t i = base + j * kWave;
        e[j] = i < a.n ? a.ids[i] : kNone;
    }
    for (uint32_t x = lane; x < a.experts; x += kWave) s_count[x] = 0;
    if (SOURCE == kTileCounts) {
        // chunk c of 64 experts and slice q of the tiles for each wave
        const uint32_t chunks = (a.experts + kWave - 1) / kWave;
        const uint32_t slices = kGroupWaves / chunks;
        const uint32_t c = wave % chunks, q = wave / chunks;
        const uint32_t x = c * kWave + lane;
        uint32_t before = 0, all = 0;
        if (q < slices && x < a.experts) {
            constexpr uint32_t kAhead = 8;   // loads in flight: of the last tile again behind the end
            for (uint32_t t0 = q; t0 < gridDim.x; t0 += kAhead * slices) {
                uint32_t n[kAhead];
#pragma unroll
                for (uint32_t j = 0; j < kAhead; ++j) {
                    const uint32_t t = t0 + j * slices;
                    n[j] = tile_counts[static_cast<uint64_t>(t < gridDim.x ? t : gridDim.x - 1) * a.experts + x];
                }
#pragma unroll
                for (uint32_t j = 0; j < kAhead; ++j) {
                    const uint32_t t = t0 + j * slices;
                    all += t < gridDim.x ? n[j] : 0u;
                    before += t < tile ? n[j] : 0u;
                }
            }
        }
        s_part[0][tid] = before;
        s_part[1][tid] = all;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const bool real = e[j] < a.experts;
        uint64_t peers = ballot(real);
        for (uint32_t b = 0; b < bits; ++b) {
            const uint64_t ones = ballot((e[j] >> b) & 1u);
            peers &= ((e[j] >> b) & 1u) ? ones : ~ones;
        }
        const uint32_t below = count_below(peers);
        rank[j] = real ? s_count[e[j]] + below : 0u;
        wave_fence();   // all peers have read before the last of them writes
        if (real && below + 1 == static_cast<uint32_t>(__builtin_popcountll(peers)))
            s_count[e[j]] = static_cast<uint16_t>(rank[j] + 1);
        wave_fence();
    }
    __syncthreads();
    uint32_t before = 0, total = 0;
    if (tid < a.experts) {
        uint16_t* column = reinterpret_cast<uint16_t*>(s_end + a.experts) + tid;
        uint32_t sum = 0;
#pragma unroll
        for (uint32_t w = 0; w < kGroupWaves; ++w) {
            const uint32_t n = column[w * a.experts];
            column[w * a.experts] = static_cast<uint16_t>(sum);
            sum += n;
        }
        total = sum;
        if (SOURCE == kTileCounts) {
            const uint32_t chunks = (a.experts + kWave - 1) / kWave;
            total = 0;
            for (uint32_t q = 0; q < kGroupWaves / chunks; ++q) {
                before += s_part[0][q * chunks * kWave + tid];
                total += s_part[1][q * chunks * kWave + tid];
            }
        } else if (SOURCE == kTileOffsets) {
            before = tile_counts[static_cast<uint64_t>(tile) * a.experts + tid];
            total = totals[tid];
        }
    }
    // the segments: padded totals, summed over the experts
    const uint32_t padded = (total + a.align - 1) / a.align * a.align;
    const uint32_t incl = wave_inclusive_sum(padded);
    if (lane == kWave - 1) s_wave[wave] = incl;
    __syncthreads();
    uint32_t start = incl - padded;
    for (uint32_t w = 0; w < wave; ++w) start += s_wave[w];
    if (tid < a.experts) {
        s_base[tid] = start + before;
        s_pad[tid] = start + total;
        s_end[tid] = start + padded;
        if (tid == a.experts - 1) s_length = start + padded;
        if (tile == 0) {
            a.counts[tid] = total;
            a.starts[tid] = start;
            if (tid == a.experts - 1) a.starts[a.experts] = start + padded;
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const uint32_t i = base + j * kWave;
        uint32_t at = kNone;
        if (e[j] < a.experts) {
            at = s_base[e[j]] + s_count[e[j]] + rank[j];
            a.order[at] = i;
        }
        if (i < a.n) a.place[i] = at;
    }
    // the padding, a wave for each expert, and the room behind the last segment
    if (a.align > 1) {
        for (uint32_t x = tile * kGroupWaves + wave; x < a.experts; x += gridDim.x * kGroupWaves)
            for (uint32_t p = s_pad[x] + lane; p < s_end[x]; p += kWave) a.order[p] = kNone;
    }
    for (uint32_t p = s_length + tile * kGroupBlock + tid; p < a.room; p += gridDim.x * kGroupBlock) a.order[p] = kNone;
}

template <int ITEMS>
hipError_t group_items_of(const GroupArgs& a, uint32_t tiles, uint32_t* temp, hipStream_t stream) {
    uint32_t bits = 0;
    while ((1u << bits) < a.experts) ++bits;
    const size_t lds = a.experts * (3 * sizeof(uint32_t) + kGroupWaves * sizeof(uint16_t));
    const uint64_t counts = static_cast<uint64_t>(tiles) * a.experts;
    hipError_t e = hipSuccess;
    if (tiles > 1) {
        timing_before(stream, RS_KERNEL_GROUP_COUNT);
        group_count_kernel<ITEMS><<<dim3(tiles), kGroupBlock, 0, stream>>>(a, temp);
        e = hipGetLastError();
        timing_after(stream);
        if (e != hipSuccess) return e;
    }
    uint32_t* totals = temp + counts;
    if (tiles > 1 && counts > kShortSum) {
        timing_before(stream, RS_KERNEL_GROUP_SCAN);
        group_scan_kernel<<<dim3((a.experts + kScanExperts - 1) / kScanExperts), kGroupBlock, 0, stream>>>(a.experts, tiles, temp, totals);
        e = hipGetLastError();
        timing_after(stream);
        if (e != hipSuccess) return e;
    }
    timing_before(stream, RS_KERNEL_GROUP_PLACE);
    const auto kernel = tiles <= 1 ? group_place_kernel<ITEMS, kAlone>
                        : counts > kShortSum ? group_place_kernel<ITEMS, kTileOffsets>
                                             : group_place_kernel<ITEMS, kTileCounts>;
    kernel<<<dim3(tiles ? tiles : 1), kGroupBlock, lds, stream>>>(a, bits, temp, totals);
    e = hipGetLastError();
    timing_after(stream);
    return e;
}

}  // namespace

size_t group_temp_bytes(uint64_t n, uint32_t experts) {
    const uint64_t tiles = group_tiles(n);
    return tiles > 1 ? (tiles + 1) * experts * sizeof(uint32_t) : RS_NO_TEMP;
}

hipError_t launch_group(const GroupArgs& a, void* temp, hipStream_t stream) {
    const uint32_t tiles = group_tiles(a.n);
    uint32_t* words = static_cast<uint32_t*>(temp);
    return group_items(a.n) == 1 ? group_items_of<1>(a, tiles, words, stream)
                                 : group_items_of<4>(a, tiles, words, stream);
}

}  // namespace rs
