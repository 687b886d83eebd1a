// group_kernels.hpp -- gfx950 (CDNA4, wave64) kernels that order ids stably: one
// counting pass for a grouping by expert, one to four for an embedding's ids (of up to
// eleven bits each, by the number of ids and of rows).
//
// Few ids are ordered here, up to a million: their bytes are nothing (12 to 20 per
// id), so launches and dependent steps bound them.  A pass is one launch (a block
// counts and places, and counts the other blocks' ids too) or two (count, place), and
// an embedding's few thousand ids take all their passes in one launch of one block.
// 1024 threads a block: 16 waves rank 64 ids each by ballots, and the counts of the
// waves before are summed bin by bin.  32 ids of 128 groups take 3.1 us (the kernel
// alone), 4,096 of 256 groups 5.6, 131,072 11.4 (calls back to back in a captured graph);
// the launch itself is some 2 us of each.  Larger orders take the library's sort.
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
    int n;
    uint32_t mask;
    uint16_t bins;
    uint8_t shift, bits;
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

// Adds the active lanes' digits to the counts in LDS.  Lanes of the last bin (of no
// group: most of them, for a rank's share of the experts) add once together, and so
// does a wave whose others are all of one bin: 64 adds to one word would queue.
__device__ __forceinline__ void count_digit(uint32_t *count, uint32_t digit, uint32_t last)
{
    if (digit == last) {
        const uint64_t on = __ballot(1);
        if (lanes_below(on) == 0) atomicAdd(&count[last], (uint32_t)__popcll(on));
    } else {
        const uint32_t f = __builtin_amdgcn_readfirstlane(digit);
        if (__ballot(digit != f) == 0) {
            const uint64_t on = __ballot(1);
            if (lanes_below(on) == 0) atomicAdd(&count[f], (uint32_t)__popcll(on));
        } else {
            atomicAdd(&count[digit], 1u);
        }
    }
}

// Digit counts of block b = slots [b * 1024 * ITEMS, ...), one row of `bins` each.
// `clear`, where given, is a word set to zero for a later kernel.
template <typename SRC, int MAX_BINS, int ITEMS>
__global__ __launch_bounds__(kPlaceThreads) void count_kernel(SRC src, Pass ps, uint32_t *__restrict__ counts,
                                                              uint32_t *clear)
{
    if (clear != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *clear = 0;
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
        if (first + i * kPlaceThreads < ps.n) count_digit(s_count, d[i], ps.bins - 1);
    }
    __syncthreads();
    uint32_t *mine = counts + (int64_t)blockIdx.x * ps.bins;
    for (uint32_t b = threadIdx.x; b < ps.bins; b += kPlaceThreads) mine[b] = s_count[b];
}

// LDS of a placement by 1024 threads.
template <int MAX_BINS>
struct PlaceSmem {
    uint32_t wave[kPlaceWaves * MAX_BINS];  // per wave: counts, then the slots of earlier waves
    uint32_t all[MAX_BINS], start[MAX_BINS];
    uint32_t tmp[kPlaceWaves];
};

// Places of a block's slots, slot i of lane l of wave w being the block's
// w * 64 * ITEMS + i * 64 + l, `valid` or not: a slot's place is its bin's start, plus
// the bin's slots in earlier blocks, in earlier waves of the block and before it in
// its wave.  `counts` holds every block's digit counts; where it is NULL, a block
// counts the other blocks' slots itself (`other` gives a slot's key).  Every thread
// calls it.
template <int MAX_BINS, int ITEMS, typename KEY>
__device__ __forceinline__ void place_slots(const Pass &ps, const uint32_t (&key)[ITEMS], const bool (&valid)[ITEMS],
                                            const uint32_t *__restrict__ counts, int block, int blocks, KEY other,
                                            int32_t *offsets, PlaceSmem<MAX_BINS> &s, uint32_t (&to)[ITEMS])
{
    constexpr int PER = (MAX_BINS + kPlaceThreads - 1) / kPlaceThreads;
    const int tid = threadIdx.x, wave = tid >> 6;
    for (uint32_t b = tid; b < kPlaceWaves * ps.bins; b += kPlaceThreads) s.wave[b] = 0;
    for (uint32_t b = tid; b < ps.bins; b += kPlaceThreads) s.all[b] = 0, s.start[b] = 0;
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
                before += r < block ? c : 0u;
            }
            atomicAdd(&s.all[b], all);
            atomicAdd(&s.start[b], before);
        }
    } else if (blocks > 1) {
        constexpr int AHEAD = 4;
        const int64_t mine = (int64_t)block * kPlaceThreads * ITEMS, after = mine + kPlaceThreads * ITEMS;
        for (int64_t at = tid; at < ps.n; at += AHEAD * kPlaceThreads) {
            uint32_t d[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (at + u * kPlaceThreads < ps.n) d[u] = digit_in(ps, other(at + u * kPlaceThreads));
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                // (a wave's 64 slots are all before this block's, in it, or after)
                const int64_t i = at + u * kPlaceThreads;
                if (i < ps.n && (i < mine || i >= after)) count_digit(i < mine ? s.start : s.all, d[u], ps.bins - 1);
            }
        }
    }
    uint32_t rank[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        rank[i] = wave_rank(valid[i] ? digit_in(ps, key[i]) : 0u, valid[i], ps.bits, s.wave + wave * ps.bins);
    __syncthreads();
    for (uint32_t b = tid; b < ps.bins; b += kPlaceThreads) {
        uint32_t sum = 0;
#pragma unroll
        for (int w = 0; w < kPlaceWaves; ++w) {
            const uint32_t c = s.wave[w * ps.bins + b];
            s.wave[w * ps.bins + b] = sum;
            sum += c;
        }
        // (counted here: the bin's slots before this block, in it, and after it)
        if (counts == nullptr) s.all[b] += s.start[b] + sum;
    }
    __syncthreads();
    uint32_t mine[PER], total = 0;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const uint32_t b = tid * PER + q;
        mine[q] = b < ps.bins ? s.all[b] : 0u;
        total += mine[q];
    }
    uint32_t start = place_scan(total, s.tmp);
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const uint32_t b = tid * PER + q;
        if (b < ps.bins) {
            s.start[b] += start;
            if (offsets != nullptr && block == 0) offsets[b] = (int32_t)start;
        }
        start += mine[q];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        if (valid[i]) {
            const uint32_t d = digit_in(ps, key[i]);
            to[i] = s.start[d] + s.wave[wave * ps.bins + d] + rank[i];
        }
}

// One block's share of a pass: slots [block * 1024 * ITEMS, ...).
template <typename SRC, int MAX_BINS, int ITEMS>
__global__ __launch_bounds__(kPlaceThreads) void place_kernel(SRC src, Pass ps, const uint32_t *__restrict__ counts,
                                                              int blocks, PlaceOut out, uint32_t *clear)
{
    if (clear != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *clear = 0;
    __shared__ PlaceSmem<MAX_BINS> s;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t first = (int64_t)blockIdx.x * kPlaceThreads * ITEMS + wave * 64 * ITEMS + lane;
    uint32_t key[ITEMS], to[ITEMS];
    bool valid[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        valid[i] = first + i * 64 < ps.n;
        if (valid[i]) key[i] = src.key(first + i * 64);
    }
    place_slots<MAX_BINS, ITEMS>(ps, key, valid, counts, blockIdx.x, blocks, [&](int64_t i) { return src.key(i); },
                                 out.offsets, s, to);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        if (!valid[i]) continue;
        const int64_t at = first + i * 64;
        if (out.keys != nullptr) out.keys[to[i]] = key[i];
        if (out.values != nullptr) out.values[to[i]] = src.value(at);
        if (out.position != nullptr) out.position[at] = digit_in(ps, key[i]) + 1 < ps.bins ? (int32_t)to[i] : -1;
    }
}

// The whole order of up to 1024 * ITEMS ids by one block: pass after pass of
// `digit_bits` bits from the lowest, the pairs kept in LDS between them.
template <typename ID, int MAX_BINS, int ITEMS>
__global__ __launch_bounds__(kPlaceThreads) void order_kernel(IdSource<ID> src, int n, int bits, int digit_bits,
                                                              uint32_t *__restrict__ sorted,
                                                              uint32_t *__restrict__ index, uint32_t *clear)
{
    if (clear != nullptr && threadIdx.x == 0) *clear = 0;
    __shared__ PlaceSmem<MAX_BINS> s;
    __shared__ uint32_t s_key[kPlaceThreads * ITEMS], s_value[kPlaceThreads * ITEMS];
    const int first = (threadIdx.x >> 6) * 64 * ITEMS + (threadIdx.x & 63);
    uint32_t key[ITEMS], value[ITEMS], to[ITEMS];
    bool valid[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        valid[i] = first + i * 64 < n;
        value[i] = (uint32_t)(first + i * 64);
        if (valid[i]) key[i] = src.key(first + i * 64);
    }
    for (int shift = 0; shift < bits; shift += digit_bits) {
        const int width = digit_bits < bits - shift ? digit_bits : bits - shift;
        const Pass ps{n, (1u << width) - 1u, (uint16_t)(1u << width), (uint8_t)shift, (uint8_t)width};
        place_slots<MAX_BINS, ITEMS>(ps, key, valid, nullptr, 0, 1, [](int64_t) { return 0u; }, nullptr, s, to);
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (valid[i]) s_key[to[i]] = key[i], s_value[to[i]] = value[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (valid[i]) key[i] = s_key[first + i * 64], value[i] = s_value[first + i * 64];
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        if (valid[i]) sorted[first + i * 64] = key[i], index[first + i * 64] = value[i];
}

}  // namespace lrs_rows
