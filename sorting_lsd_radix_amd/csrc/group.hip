// group.hip -- the choices of a router ordered by expert: a stable partition
// with one side for each expert.
//
// Three launches: every tile counts its choices of each expert; one block
// turns the counts into the experts' segments and every tile's offsets in
// them; every tile puts its choices in their places.  Nothing depends on the
// order in which blocks or atomics run: counts are sums, and the rank of a
// choice in its tile comes from ballots over waves that take turns.
#include "internal.hpp"
#include "device_common.hpp"

namespace rs {

namespace {

constexpr int kGroupBlock = 256;
constexpr uint32_t kGroupTile = 4096;        // smallest tile
constexpr uint32_t kGroupMaxTiles = 1024;
constexpr uint32_t kNone = 0xFFFFFFFFu;

uint32_t group_tile(uint64_t n) {
    const uint64_t share = (n + kGroupMaxTiles - 1) / kGroupMaxTiles;
    const uint64_t tile = (share + kGroupBlock - 1) / kGroupBlock * kGroupBlock;
    return static_cast<uint32_t>(tile < kGroupTile ? kGroupTile : tile);
}

uint32_t group_tiles(uint64_t n) {
    const uint32_t tile = group_tile(n);
    return static_cast<uint32_t>((n + tile - 1) / tile);
}

__global__ __launch_bounds__(kGroupBlock) void group_count_kernel(GroupArgs a, uint32_t tile,
                                                                  uint32_t* __restrict__ tile_counts) {
    __shared__ uint32_t s_count[RS_MAX_EXPERTS];
    for (uint32_t e = threadIdx.x; e < a.experts; e += kGroupBlock) s_count[e] = 0;
    __syncthreads();
    const uint32_t base = blockIdx.x * tile;
    const uint32_t end = a.n - base < tile ? a.n : base + tile;
    for (uint32_t i = base + threadIdx.x; i < end; i += kGroupBlock) {
        const uint32_t e = a.ids[i];
        if (e < a.experts) atomicAdd(&s_count[e], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.experts; e += kGroupBlock)
        tile_counts[static_cast<uint64_t>(blockIdx.x) * a.experts + e] = s_count[e];
}

// One block, thread e for expert e: tile_counts become the choices of earlier
// tiles, and the totals the padded segments.
__global__ __launch_bounds__(RS_MAX_EXPERTS) void group_scan_kernel(GroupArgs a, uint32_t tiles,
                                                                    uint32_t* __restrict__ tile_counts) {
    constexpr int kWaves = RS_MAX_EXPERTS / kWave;
    __shared__ uint32_t s_wave[kWaves];
    const uint32_t e = threadIdx.x;
    uint32_t count = 0;
    if (e < a.experts) {
        for (uint32_t t = 0; t < tiles; ++t) {
            uint32_t* c = &tile_counts[static_cast<uint64_t>(t) * a.experts + e];
            const uint32_t own = *c;
            *c = count;
            count += own;
        }
    }
    const uint32_t padded = (count + a.align - 1) / a.align * a.align;
    const uint32_t incl = wave_inclusive_sum(padded);
    if ((e & (kWave - 1)) == kWave - 1) s_wave[e / kWave] = incl;
    __syncthreads();
    uint32_t before = 0;
    for (uint32_t w = 0; w < e / kWave; ++w) before += s_wave[w];
    if (e < a.experts) {
        a.counts[e] = count;
        a.starts[e] = before + incl - padded;
        if (e == a.experts - 1) a.starts[a.experts] = before + incl;
    }
}

__global__ __launch_bounds__(kGroupBlock) void group_place_kernel(GroupArgs a, uint32_t tile,
                                                                  const uint32_t* __restrict__ tile_counts) {
    __shared__ uint32_t s_next[RS_MAX_EXPERTS];
    const uint32_t tid = threadIdx.x;
    for (uint32_t e = tid; e < a.experts; e += kGroupBlock)
        s_next[e] = a.starts[e] + (a.n ? tile_counts[static_cast<uint64_t>(blockIdx.x) * a.experts + e] : 0u);
    __syncthreads();
    const uint32_t wave = tid / kWave;
    const uint32_t base = blockIdx.x * tile;
    const uint32_t end = a.n - base < tile ? a.n : base + tile;
    for (uint32_t i0 = base; i0 < end; i0 += kGroupBlock) {
        const uint32_t i = i0 + tid;
        const uint32_t e = i < end ? a.ids[i] : kNone;
        const bool real = e < a.experts;
        uint64_t same = ballot(real);
        for (int b = 0; b < 10; ++b) {
            const uint64_t ones = ballot((e >> b) & 1u);
            same &= ((e >> b) & 1u) ? ones : ~ones;
        }
        const uint32_t rank = count_below(same);
        uint32_t at = kNone;
        for (uint32_t w = 0; w < kGroupBlock / kWave; ++w) {   // the waves take turns, in order
            if (w == wave && real) {
                at = s_next[e] + rank;
                // every lane of the expert has read the word before the last of them writes it
                __builtin_amdgcn_wave_barrier();
                if (rank + 1 == static_cast<uint32_t>(__builtin_popcountll(same))) s_next[e] = at + 1;
            }
            __syncthreads();
        }
        if (real) a.order[at] = i;
        if (i < end) a.place[i] = at;
    }
    // the padding, and the room behind the last segment
    for (uint32_t e = blockIdx.x; e < a.experts; e += gridDim.x)
        for (uint32_t p = a.starts[e] + a.counts[e] + tid; p < a.starts[e + 1]; p += kGroupBlock) a.order[p] = kNone;
    for (uint32_t p = a.starts[a.experts] + blockIdx.x * kGroupBlock + tid; p < a.room; p += gridDim.x * kGroupBlock)
        a.order[p] = kNone;
}

}  // namespace

size_t group_temp_bytes(uint64_t n, uint32_t experts) {
    const size_t words = static_cast<size_t>(group_tiles(n)) * experts;
    return (words ? words : 1) * 4;
}

hipError_t launch_group(const GroupArgs& a, void* temp, hipStream_t stream) {
    uint32_t* tile_counts = static_cast<uint32_t*>(temp);
    const uint32_t tile = group_tile(a.n), tiles = group_tiles(a.n);
    if (tiles) {
        timing_before(stream, RS_KERNEL_GROUP_COUNT);
        group_count_kernel<<<dim3(tiles), kGroupBlock, 0, stream>>>(a, tile, tile_counts);
        const hipError_t e = hipGetLastError();
        timing_after(stream);
        if (e != hipSuccess) return e;
    }
    timing_before(stream, RS_KERNEL_GROUP_SCAN);
    group_scan_kernel<<<dim3(1), RS_MAX_EXPERTS, 0, stream>>>(a, tiles, tile_counts);
    hipError_t e = hipGetLastError();
    timing_after(stream);
    if (e != hipSuccess) return e;
    timing_before(stream, RS_KERNEL_GROUP_PLACE);
    group_place_kernel<<<dim3(tiles ? tiles : 1), kGroupBlock, 0, stream>>>(a, tile, tile_counts);
    e = hipGetLastError();
    timing_after(stream);
    return e;
}

}  // namespace rs
