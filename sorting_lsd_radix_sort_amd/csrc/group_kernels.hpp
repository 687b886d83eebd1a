// group_kernels.hpp -- gfx950 (CDNA4, wave64) kernels that order ids stably: one
// counting pass for a grouping by expert, two or three for an embedding's ids.
//
// Few ids are ordered here, up to some hundred thousand: their bytes are nothing, so
// launches and dependent steps bound them, and each pass runs in one launch of one
// workgroup or in two launches (count, place) of a few.  Larger orders take the
// library's sort.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lrs_rows {

constexpr int kPlaceThreads = 1024;
constexpr int kPlaceWaves = kPlaceThreads / 64;

// Where keys and the indices that travel with them come from.
//
// An id's key is id - first where that is below `groups`, else `groups`: those of no
// group come last.
template <typename ID>
struct IdSource {
    const ID *__restrict__ ids;
    int64_t first;
    uint32_t groups;
    __device__ __forceinline__ uint32_t key(int64_t i) const
    {
        const uint64_t g = (uint64_t)ids[i] - (uint64_t)first;
        return g < groups ? (uint32_t)g : groups;
    }
    __device__ __forceinline__ uint32_t value(int64_t i) const { return (uint32_t)i; }
};

// The pairs that an earlier pass left.
struct PairSource {
    const uint32_t *__restrict__ keys;
    const uint32_t *__restrict__ values;
    __device__ __forceinline__ uint32_t key(int64_t i) const { return keys[i]; }
    __device__ __forceinline__ uint32_t value(int64_t i) const { return values[i]; }
};

// A pass: its digit is (key >> shift) & mask, below `bins`, which is at most 2^bits
// and a kernel's MAX_BINS.  (A grouping's last bin holds the ids of no group.)
struct Pass {
    int64_t n;
    int shift, bits;
    uint32_t mask, bins;
};

__device__ __forceinline__ uint32_t digit_in(const Pass &ps, uint32_t key) { return (key >> ps.shift) & ps.mask; }

// What a pass writes, each where it is not NULL: keys and values in order, each
// index's place (-1 in the last bin), and where each bin begins.
struct PlaceOut {
    uint32_t *keys, *values;
    int32_t *position, *offsets;
};

// Number of set bits of `lanes` below this lane.
__device__ __forceinline__ uint32_t lanes_below(uint64_t lanes)
{
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(lanes >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)lanes, 0u));
}

// Exclusive prefix sum of one value per thread over the workgroup; every thread
// calls it.
__device__ __forceinline__ uint32_t place_scan(uint32_t v, uint32_t *s_tmp)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    if (lane == 63) s_tmp[wave] = x;
    __syncthreads();
    uint32_t before = 0;
#pragma unroll
    for (int w = 0; w < kPlaceWaves; ++w) before += w < wave ? s_tmp[w] : 0u;
    return before + x - v;
}

// Rank of a key among the equal digits that this wave has seen, counted on in
// `count` (the wave's bins in LDS).  A lane's equals are the lanes whose ballot
// agrees with it in each of the digit's `bits` bits: four vector instructions a bit
// (v_bitop3 0x90 is m & ~(ballot ^ t), t all ones where the lane's own bit is set).
__device__ __forceinline__ uint32_t wave_rank(uint32_t digit, bool valid, int bits, volatile uint32_t *count)
{
    const uint64_t on = __ballot(valid);
    uint32_t lo = (uint32_t)on, hi = (uint32_t)(on >> 32);
    for (int b = 0; b < bits; ++b) {
        const uint32_t t = (uint32_t)__builtin_amdgcn_sbfe((int)digit, (uint32_t)b, 1u);
        const uint64_t set = __ballot(t != 0u);
        lo = __builtin_amdgcn_bitop3_b32(lo, (uint32_t)set, t, 0x90);
        hi = __builtin_amdgcn_bitop3_b32(hi, (uint32_t)(set >> 32), t, 0x90);
    }
    const uint64_t same = ((uint64_t)hi << 32) | lo;
    const uint32_t below = lanes_below(same);
    uint32_t rank = 0;
    if (valid) {
        const uint32_t seen = count[digit];
        rank = seen + below;
        // (a wave's LDS accesses complete in order: all lanes have read before this)
        if (below == 0) count[digit] = seen + (uint32_t)__popcll(same);
    }
    __builtin_amdgcn_wave_barrier();
    return rank;
}

// Digit counts of block b = slots [b * 1024 * ITEMS, ...), one row of `bins` each.
template <typename SRC, int MAX_BINS, int ITEMS>
__global__ __launch_bounds__(kPlaceThreads) void count_kernel(SRC src, Pass ps, uint32_t *__restrict__ counts)
{
    __shared__ uint32_t s_count[MAX_BINS];
    for (uint32_t b = threadIdx.x; b < ps.bins; b += kPlaceThreads) s_count[b] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * kPlaceThreads * ITEMS + threadIdx.x;
    uint32_t d[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        if (first + i * kPlaceThreads < ps.n) d[i] = digit_in(ps, src.key(first + i * kPlaceThreads));
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        if (first + i * kPlaceThreads < ps.n) {
            // a wave of one digit adds once: 64 adds to one word would queue
            const uint32_t f = __builtin_amdgcn_readfirstlane(d[i]);
            const uint64_t on = __ballot(1);
            if (__ballot(d[i] != f) == 0) {
                if (lanes_below(on) == 0) atomicAdd(&s_count[f], (uint32_t)__popcll(on));
            } else {
                atomicAdd(&s_count[d[i]], 1u);
            }
        }
    }
    __syncthreads();
    for (uint32_t b = threadIdx.x; b < ps.bins; b += kPlaceThreads) counts[(int64_t)blockIdx.x * ps.bins + b] = s_count[b];
}

// Stable placement of block b's slots.  `counts` holds every block's digit counts
// (from count_kernel), or is NULL for a pass of one block, which counts as it ranks.
// Each wave ranks 64 * ITEMS slots in a row; a slot's place is its bin's start, plus
// the bin's slots in earlier blocks, in earlier waves of the block and before it in
// its wave.
template <typename SRC, int MAX_BINS, int ITEMS>
__global__ __launch_bounds__(kPlaceThreads) void place_kernel(SRC src, Pass ps, const uint32_t *__restrict__ counts,
                                                              int blocks, PlaceOut out)
{
    constexpr int PER = (MAX_BINS + kPlaceThreads - 1) / kPlaceThreads;
    __shared__ uint32_t s_wave[kPlaceWaves * MAX_BINS];  // per wave: counts, then the slots of earlier waves
    __shared__ uint32_t s_all[MAX_BINS], s_start[MAX_BINS];
    __shared__ uint32_t s_tmp[kPlaceWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t first = (int64_t)blockIdx.x * kPlaceThreads * ITEMS + wave * 64 * ITEMS + lane;
    uint32_t key[ITEMS], rank[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        if (first + i * 64 < ps.n) key[i] = src.key(first + i * 64);
    for (uint32_t b = tid; b < kPlaceWaves * ps.bins; b += kPlaceThreads) s_wave[b] = 0;
    for (uint32_t b = tid; b < ps.bins; b += kPlaceThreads) s_all[b] = 0, s_start[b] = 0;
    __syncthreads();
    if (counts != nullptr) {
        // each bin's slots in all blocks and in earlier ones: 1024 / bins lanes per
        // bin (a power of two) share its rows
        int width = 1;
        while (width < (int)ps.bins && width < kPlaceThreads) width *= 2;
        const int parts = kPlaceThreads / width, part = tid / width;
        for (uint32_t b = tid & (width - 1); b < ps.bins; b += width) {
            uint32_t all = 0, before = 0;
#pragma unroll 8
            for (int r = part; r < blocks; r += parts) {
                const uint32_t c = counts[(int64_t)r * ps.bins + b];
                all += c;
                before += r < (int)blockIdx.x ? c : 0u;
            }
            atomicAdd(&s_all[b], all);
            atomicAdd(&s_start[b], before);
        }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const bool valid = first + i * 64 < ps.n;
        rank[i] = wave_rank(valid ? digit_in(ps, key[i]) : 0u, valid, ps.bits, s_wave + wave * ps.bins);
    }
    __syncthreads();
    for (uint32_t b = tid; b < ps.bins; b += kPlaceThreads) {
        uint32_t sum = 0;
#pragma unroll
        for (int w = 0; w < kPlaceWaves; ++w) {
            const uint32_t c = s_wave[w * ps.bins + b];
            s_wave[w * ps.bins + b] = sum;
            sum += c;
        }
        if (counts == nullptr) s_all[b] = sum;
    }
    __syncthreads();
    uint32_t mine[PER], total = 0;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const uint32_t b = tid * PER + q;
        mine[q] = b < ps.bins ? s_all[b] : 0u;
        total += mine[q];
    }
    uint32_t start = place_scan(total, s_tmp);
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const uint32_t b = tid * PER + q;
        if (b < ps.bins) {
            s_start[b] += start;
            if (out.offsets != nullptr && blockIdx.x == 0) out.offsets[b] = (int32_t)start;
        }
        start += mine[q];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int64_t at = first + i * 64;
        if (at < ps.n) {
            const uint32_t d = digit_in(ps, key[i]);
            const uint32_t to = s_start[d] + s_wave[wave * ps.bins + d] + rank[i];
            if (out.keys != nullptr) out.keys[to] = key[i];
            if (out.values != nullptr) out.values[to] = src.value(at);
            if (out.position != nullptr) out.position[at] = d + 1 < ps.bins ? (int32_t)to : -1;
        }
    }
}

}  // namespace lrs_rows
