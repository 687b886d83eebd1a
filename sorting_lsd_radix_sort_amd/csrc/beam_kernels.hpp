// beam_kernels.hpp -- gfx950 (CDNA4, wave64) kernels of beam search
// (include/lrsort_choose.h): the best continuations over all beams and the vocabulary,
// and the beams' states put in the order of their parents.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "choose_common.hpp"

namespace lrs_choose {

constexpr int kScanThreads = 256, kScanWaves = kScanThreads / kWave;
constexpr int kMaxContinuations = 64, kMaxBeams = 1024;  // of one search
constexpr int kHeld = 2 * kWave;   // candidates that a wave holds

// A candidate is its logit's order key above the complement of its token: larger is
// better, and of equal logits the lowest token.
__device__ __forceinline__ uint64_t candidate_of(float l, int token)
{
    return (uint64_t)key_of(l) << 32 | (uint32_t)~token;
}

__device__ __forceinline__ float logit_of(uint64_t c) { return value_of((uint32_t)(c >> 32)); }
__device__ __forceinline__ int token_of(uint64_t c) { return (int)~(uint32_t)c; }

// What a wave leaves of its part of a row beside its best candidates: the largest logit
// and the sum of exp(l - top).
struct Part {
    double sum;
    float top;
    float pad;
};

// Of the first `n` <= kHeld candidates in LDS keeps the `count` best, in order, and
// returns how many these are.
__device__ __forceinline__ int keep_best(uint64_t *held, int n, int count, int lane)
{
    wave_sync();
    const uint64_t a = lane < n ? held[lane] : 0ull, b = lane + kWave < n ? held[lane + kWave] : 0ull;
    int before_a = 0, before_b = 0;
    for (int i = 0; i < n; ++i) {
        const uint64_t o = held[i];
        before_a += o > a;
        before_b += o > b;
    }
    wave_sync();
    if (lane < n && before_a < count) held[before_a] = a;
    if (lane + kWave < n && before_b < count) held[before_b] = b;
    wave_sync();
    return n < count ? n : count;
}

struct Scan {
    const float *scores;
    const uint8_t *finished;
    uint64_t *best;  // rows x parts x count
    Part *of_part;   // rows x parts
    int64_t part;    // logits of one, a multiple of a wave's step
    int rows, vocab, parts, count;
};

// A wave reads its part of a row once, 16 bytes a lane at a time, keeping the `count`
// best logits and (SUM) the maximum and the sum of the softmax.  A logit becomes a
// candidate where it is above the worst kept one; of the first step's logits those that
// the `count`-th of the lanes' maxima does not exceed.
template <typename T, bool SUM>
__global__ __launch_bounds__(kScanThreads) void beam_scan_kernel(const T *__restrict__ logits, int64_t ld, Scan a)
{
    constexpr int VEC = kVec<T>, STEP = kWave * VEC;
    __shared__ uint64_t of_wave[kScanWaves][kHeld];
    const int lane = (int)threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    uint64_t *held = of_wave[wave];
    const float none = -__builtin_inff();

    const int64_t jobs = (int64_t)a.rows * a.parts;
    for (int64_t job = (int64_t)blockIdx.x * kScanWaves + wave; job < jobs; job += kMaxGridX * kScanWaves) {
        const int row_at = (int)(job / a.parts);
        // (64 bits: a step past the end of a vocabulary of 2^31 - 1 is no int)
        const int64_t from = job % a.parts * a.part;
        const int64_t to = a.vocab - from < a.part ? a.vocab : from + a.part;
        const float score = a.scores[row_at];
        if (score == none || (a.finished != nullptr && a.finished[row_at] != 0)) continue;
        const T *row = logits + row_at * ld;

        int n = 0;                // held
        uint64_t above = 0ull;    // a candidate is larger
        float least = none;       // and its logit not below this
        float top = none;
        double sum = 0.0;
        bool first = true;
        for (int64_t c0 = from; c0 < to; c0 += STEP) {
            const Col col = col_of<T>(to, c0 + lane * VEC);
            const u32x4 r = load_col<T, true>(row, col);
            float l[VEC];
            float most = none;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                l[i] = i < col.valid ? element<T>(r, i) : none;
                most = __builtin_fmaxf(most, l[i]);
            }
            if constexpr (SUM) {
                const float higher = __builtin_fmaxf(top, most);
                if (higher != none) {
                    float part = 0.0f;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) part += __builtin_amdgcn_exp2f((l[i] - higher) * 1.44269504f);
                    sum = sum * (double)__builtin_amdgcn_exp2f((top - higher) * 1.44269504f) + (double)part;
                    top = higher;
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (l[i] != l[i]) sum += (double)l[i];  // NaN beside nothing but -infinity
                }
            }
            if (first) {
                // at least `count` logits are not below the count-th largest maximum
                const uint32_t mine = key_of(most);
                int before = 0;
                for (int i = 0; i < kWave; ++i) {
                    const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)mine, i);
                    before += o > mine || (o == mine && i < lane);
                }
                const uint64_t there = __builtin_amdgcn_ballot_w64(before == a.count - 1);
                const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)mine, __builtin_ctzll(there));
                above = key == 0u ? 0xFFFFFFFFull : ((uint64_t)key << 32) - 1;
                least = value_of(key);
                first = false;
            }
            if (__builtin_amdgcn_ballot_w64(most >= least && most != none) == 0ull) continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int token = (int)col.c + i;
                uint64_t c = candidate_of(l[i], token);
                bool takes = l[i] >= least && c > above && (uint32_t)(c >> 32) != 0u;
                uint64_t all = __builtin_amdgcn_ballot_w64(takes);
                if (all == 0ull) continue;
                if (n + __builtin_popcountll(all) > kHeld) {
                    n = keep_best(held, n, a.count, lane);
                    if (n == a.count) {
                        above = held[n - 1];
                        least = logit_of(above);
                    }
                    takes = takes && c > above;
                    all = __builtin_amdgcn_ballot_w64(takes);
                }
                if (takes) held[n + __builtin_popcountll(all & ((1ull << lane) - 1))] = c;
                n += __builtin_popcountll(all);
            }
        }
        n = keep_best(held, n, a.count, lane);
        if (lane < a.count) a.best[job * a.count + lane] = lane < n ? held[lane] : 0ull;
        if constexpr (SUM) {
            float high = top;
#pragma unroll
            for (int d = 1; d < kWave; d *= 2) high = __builtin_fmaxf(high, __shfl_xor(high, d, kWave));
            double s = top == none ? sum : sum * exp((double)top - (double)high);
#pragma unroll
            for (int d = 1; d < kWave; d *= 2) s += __shfl_xor(s, d, kWave);
            if (lane == 0) a.of_part[job] = Part{s, high, 0.0f};
        }
        wave_sync();
    }
}

// -------------------------------------------------------------------- joining

struct Join {
    const float *scores;
    const uint8_t *finished;
    const uint64_t *best;
    const Part *of_part;
    float *out_scores;
    int32_t *parents;
    void *tokens;
    int beams, vocab, parts, count, end_id;
    uint8_t normalize, wide_ids;
};

constexpr int kJoinThreads = 1024;

// A continuation: its total's order key (float64), then its beam and token.
struct Total {
    uint64_t key;
    uint32_t flat;  // beam * vocab + token; ~0: none
};

__device__ __forceinline__ bool better(const Total &a, const Total &b)
{
    return a.key > b.key || (a.key == b.key && a.flat < b.flat);
}

// One workgroup per search: the beams' log sums from their parts, the `count`-th best
// of the parts' best as a bound, and what reaches it ranked by counting.
__global__ __launch_bounds__(kJoinThreads) void beam_join_kernel(Join a, int batch)
{
    // the candidates taken, the first `count` of them the best so far
    __shared__ uint64_t taken_key[kMaxContinuations + kJoinThreads];
    __shared__ uint32_t taken_flat[kMaxContinuations + kJoinThreads];
    __shared__ int taken;
    __shared__ uint64_t bound_key;
    __shared__ uint32_t bound_flat;
    extern __shared__ uint64_t lds[];
    double *norm = reinterpret_cast<double *>(lds);  // of each beam: what its logits are less
    const int tid = (int)threadIdx.x;
    const float none = -__builtin_inff();

    for (int64_t b = blockIdx.x; b < batch; b += kMaxGridX) {
        // a wave per beam: log of the sum over its parts
        for (int beam = tid / kWave; beam < a.beams; beam += kJoinThreads / kWave) {
            const int64_t row = b * a.beams + beam;
            const int lane = tid % kWave;
            const float score = a.scores[row];
            const bool over = a.finished != nullptr && a.finished[row] != 0;
            double less = 0.0;
            if (a.normalize && score != none && !over) {
                float high = none;
                for (int p = lane; p < a.parts; p += kWave)
                    high = __builtin_fmaxf(high, a.of_part[row * a.parts + p].top);
#pragma unroll
                for (int d = 1; d < kWave; d *= 2) high = __builtin_fmaxf(high, __shfl_xor(high, d, kWave));
                double sum = 0.0;
                for (int p = lane; p < a.parts; p += kWave) {
                    const Part q = a.of_part[row * a.parts + p];
                    sum += q.top == none ? q.sum : q.sum * exp((double)q.top - (double)high);
                }
#pragma unroll
                for (int d = 1; d < kWave; d *= 2) sum += __shfl_xor(sum, d, kWave);
                less = (double)high + log(sum);
            }
            if (lane == 0) norm[beam] = less;
        }
        if (tid == 0) taken = 0, bound_key = 0ull, bound_flat = ~0u;
        __syncthreads();

        auto total_of = [&](int beam, uint64_t c) -> Total {
            if ((uint32_t)(c >> 32) == 0u) return {0ull, ~0u};
            const double l = (double)logit_of(c);
            const double score = (double)a.scores[b * a.beams + beam];
            return {key_of(score + (l - norm[beam])), (uint32_t)(beam * a.vocab + token_of(c))};
        };
        // list i: part i % parts of beam i / parts, its best first; the last `beams`
        // lists hold a finished beam's only continuation
        const int lists = a.beams * a.parts;
        auto candidate = [&](int list, int k) -> Total {
            if (list >= lists) {
                const int beam = list - lists;
                const int64_t row = b * a.beams + beam;
                const float score = a.scores[row];
                if (k > 0 || a.finished == nullptr || a.finished[row] == 0 || score == none) return {0ull, ~0u};
                return {key_of((double)score), (uint32_t)(beam * a.vocab + a.end_id)};
            }
            const int beam = list / a.parts;
            const int64_t row = b * a.beams + beam;
            if (a.scores[row] == none || (a.finished != nullptr && a.finished[row] != 0)) return {0ull, ~0u};
            return total_of(beam, a.best[(b * lists + list) * a.count + k]);
        };

        // The best of every list first: the `count`-th of them bounds what the others have
        // to beat.  Then the rest, every list's k-th before any list's next, in blocks of
        // as many as the workgroup has threads.  What is not better than the bound so far
        // is left out; a block of which nothing is taken, and in which every list stood,
        // is the last, since lists get worse.
        const int everything = lists + (a.finished != nullptr ? a.beams : 0);
        const int64_t all = (int64_t)everything * a.count;
        for (int64_t from = 0; from < all;) {
            const int64_t to = from < everything ? everything : all;
            const int64_t at = from + tid;
            Total t{0ull, ~0u};
            if (at < to) t = candidate((int)(at % everything), (int)(at / everything));
            const bool takes = t.key != 0ull && better(t, Total{bound_key, bound_flat});
            if (takes) {
                const int slot = atomicAdd(&taken, 1);
                taken_key[slot] = t.key, taken_flat[slot] = t.flat;
            }
            const int more = __syncthreads_or(takes);
            if (!more && from >= everything && everything <= kJoinThreads) break;
            from = from + kJoinThreads < to ? from + kJoinThreads : to;
            if (!more) continue;
            const int n = taken;
            Total mine[2];  // ranked by counting, at most two a thread
            int before[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int slot = tid + i * kJoinThreads;
                mine[i] = slot < n ? Total{taken_key[slot], taken_flat[slot]} : Total{0ull, ~0u};
            }
            if (tid < n)
                for (int o = 0; o < n; ++o) {
                    const Total other{taken_key[o], taken_flat[o]};
                    before[0] += better(other, mine[0]);
                    before[1] += better(other, mine[1]);
                }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (tid + i * kJoinThreads < n && before[i] < a.count) {
                    taken_key[before[i]] = mine[i].key, taken_flat[before[i]] = mine[i].flat;
                    if (before[i] == a.count - 1) bound_key = mine[i].key, bound_flat = mine[i].flat;
                }
            if (tid == 0) taken = n < a.count ? n : a.count;
            __syncthreads();
        }
        for (int k = tid; k < a.count; k += kJoinThreads) {
            const int64_t at = b * a.count + k;
            const bool there = k < taken;
            const uint32_t flat = there ? taken_flat[k] : 0u;
            a.out_scores[at] = there ? (float)value_of(taken_key[k]) : none;
            a.parents[at] = there ? (int32_t)(flat / (uint32_t)a.vocab) : -1;
            const int token = there ? (int)(flat % (uint32_t)a.vocab) : -1;
            if (a.wide_ids)
                ((int64_t *)a.tokens)[at] = token;
            else
                ((int32_t *)a.tokens)[at] = token;
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------- reordering

struct Places {
    int64_t outer_step, batch_step, beam_step, middle_step, row_step;
};

struct Reorder {
    const int32_t *parents;
    int64_t row_bytes, vecs;  // vecs: columns of a row
    int all_rows, rows, middle, batch, beams, count, tx_log2;
    bool in_place;
};

typedef uint32_t u32x4_byte __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32_byte __attribute__((aligned(1)));
typedef uint16_t u16_byte __attribute__((aligned(1)));

// A lane moves one column, of 16 bytes or (at a row's end) of one word, of all beams of
// a search: it has read what it needs of the old states before it stores the first of
// the new ones, so they may be the same memory.
template <typename W, int MOST>
__device__ __forceinline__ void move_column(const char *in, char *out, const Places &from, const Places &to,
                                            const int32_t *parents, int beams, int count, bool in_place)
{
    W v[MOST];
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
        v[j] = W{};
        if (j >= count) continue;
        const int p = parents[j];
        if ((uint32_t)p < (uint32_t)beams && !(in_place && p == j))
            v[j] = *reinterpret_cast<const W *>(in + p * from.beam_step);
    }
#pragma unroll
    for (int j = 0; j < MOST; ++j)
        if (j < count && !(in_place && parents[j] == j)) *reinterpret_cast<W *>(out + j * to.beam_step) = v[j];
}

// WORD: bytes of the words that a row's last columns are moved in; MOST: beams whose
// columns a lane holds at once (more of them one after another, not in place).
template <int WORD, int MOST, bool WAVE_ROW>
__global__ __launch_bounds__(kThreads) void reorder_kernel(const char *in, char *out, Places from, Places to, Reorder a)
{
    for (int64_t tile = blockIdx.y; tile << (kThreadsLog2 - a.tx_log2) < a.all_rows; tile += kMaxGridY) {
        const int64_t r64 = row_of<WAVE_ROW>(a.tx_log2, tile);
        if (r64 >= a.all_rows) continue;
        const uint32_t r = (uint32_t)r64;
        const uint32_t block = r / (uint32_t)a.rows, row = r % (uint32_t)a.rows;
        const uint32_t state = block / (uint32_t)a.middle, middle = block % (uint32_t)a.middle;
        const uint32_t outer = state / (uint32_t)a.batch, b = state % (uint32_t)a.batch;
        const char *src =
            in + outer * from.outer_step + b * from.batch_step + middle * from.middle_step + row * from.row_step;
        char *dst = out + outer * to.outer_step + b * to.batch_step + middle * to.middle_step + row * to.row_step;
        const int64_t whole = a.row_bytes / 16;
        for (int64_t x = blockIdx.x; x << a.tx_log2 < a.vecs; x += kMaxGridX) {
            const int64_t vec = (x << a.tx_log2) + (threadIdx.x & ((1 << a.tx_log2) - 1));
            if (vec >= a.vecs) continue;
#pragma unroll 1
            for (int j0 = 0; j0 < a.count; j0 += MOST) {
                const int32_t *parents = a.parents + (int64_t)b * a.count + j0;
                const int most = a.count - j0 < MOST ? a.count - j0 : MOST;
                const int64_t at = vec < whole ? vec * 16 : whole * 16 + (vec - whole) * WORD;
                char *d = dst + at + j0 * to.beam_step;
                if (vec < whole)
                    move_column<u32x4_byte, MOST>(src + at, d, from, to, parents, a.beams, most, a.in_place);
                else if constexpr (WORD == 4)
                    move_column<u32_byte, MOST>(src + at, d, from, to, parents, a.beams, most, a.in_place);
                else if constexpr (WORD == 2)
                    move_column<u16_byte, MOST>(src + at, d, from, to, parents, a.beams, most, a.in_place);
                else
                    move_column<uint8_t, MOST>(src + at, d, from, to, parents, a.beams, most, a.in_place);
            }
        }
    }
}

}  // namespace lrs_choose
