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
constexpr int kListed = kScanWaves * kMaxContinuations;  // candidates that a part collects
constexpr int kQueued = 512;                             // vectors in which there are some
constexpr int kHeld = 2 * kWave;                         // and that a wave holds among ties

// A candidate is its logit's order key above the complement of its token: larger is
// better, and of equal logits the lowest token.
__device__ __forceinline__ uint64_t candidate_of(float l, uint32_t token)
{
    return (uint64_t)key_of(l) << 32 | ~token;
}

__device__ __forceinline__ float logit_of(uint64_t c) { return value_of((uint32_t)(c >> 32)); }

// What is left of a part of a row beside its best candidates: the sum of its exp(l) is
// sum * exp(base).
struct Part {
    double sum, base;
};

// 2^(l * kLog2e) is exp(l * (1 - kLog2eLess)): log2(e) rounded to float32, and what that
// takes from an exponent.
constexpr float kLog2e = 1.44269504f;
// Below this l * kLog2e - (top * kLog2e rounded) is formed by one fma: the rounding, half
// a step of the product, is part of the base, and has to leave the exponent in range.
constexpr float kOneProduct = 1e6f;
constexpr double kLn2 = 0.693147180559945309417, kLog2eLess = 1.0 - (double)kLog2e * kLn2;

// Of the first `n` <= kHeld candidates of a wave keeps the `count` best, in order, and
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
    int rows, vocab, parts, count;
};

// A workgroup takes a part of a row, R vectors a lane, which it reads once and keeps in
// registers: first the lanes' maxima; then, with the largest of them known, (SUM) the
// part's sum of exponentials and the vectors that hold candidates.  A bound for these:
// the `count`-th largest of 64 maxima, each over an equal share of the part, so that
// some 64 (1 / 64 + 1 / 63 + .. + 1 / (65 - count)) logits reach it (18 for 16, 87 for 48,
// 170 for 60, 304 for 64).  Their vectors are queued in LDS and taken apart there, a logit
// a thread.  Where they are more than the list's 256, by ties or because `count` is nearly
// 64 (a third of the parts at 63, most at 64), a wave keeps its best in a list of its own:
// 512 rows of 131,072 bf16 logits in 71 us with the join if all are equal, 31 if none; the
// scan alone 26 for 16 of them, 32 for 48, 49 for 60, 66 for 63, 82 for 64.
//
// The part's sum: exponents by base 2 relative to the part's largest logit, eight or four
// of them added in float32, the rest in float64: its logarithm is off by 5e-8 on average,
// the share of log2(e)'s rounding (1.3e-8 of a logit's distance from the largest).  These
// are fewer bits than float64 exponentials would keep, which are some twenty instructions
// of float64 a logit where these are six of float32: totals of two beams that are closer
// than their logarithms' errors may change places.
//
// Bound by HBM and by instructions about equally: 512 rows of 131,072 bf16 logits in 26
// us, 134 MB at 5.2 TB/s (22 us without the sums, which are 6 instructions a logit and
// 16 cycles of its exponential), float32 in 45 (5.9 TB/s).  66 registers a lane (what is
// taken apart for the maxima is taken apart again), 256 threads a part (512: 4 us more
// of bf16, 9 of float32; 128: 1 and 3), eight vectors a lane (four: 2 us more, two 15;
// twelve 6, sixteen 53).  A first form, which kept a list and a bound per wave, took 84.
template <typename T, bool SUM, int R>
__global__ __launch_bounds__(kScanThreads) void beam_scan_kernel(const T *__restrict__ logits, int64_t ld, Scan a)
{
    constexpr int VEC = kVec<T>;
    constexpr int64_t PART = (int64_t)kScanThreads * VEC * R;
    __shared__ uint32_t maxima[kScanWaves][kWave];
    __shared__ uint64_t list[kListed];
    __shared__ union {
        struct {
            u32x4 vector[kQueued];
            uint32_t token[kQueued];  // of a vector's first logit
        } queue;
        uint64_t of_wave[kScanWaves][kHeld];
    } held_all;
    __shared__ double sums[kScanWaves];
    __shared__ uint32_t bound, largest;
    __shared__ int listed, queued;
    const int tid = (int)threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const float none = -__builtin_inff();

    const int64_t job = blockIdx.y * kMaxGridX + blockIdx.x;
    if (job >= (int64_t)a.rows * a.parts) return;
    const int row_at = (int)(job / a.parts);
    // (64 bits: a place past the end of a vocabulary of 2^31 - 1 is no int)
    const int64_t from = job % a.parts * PART;
    const float score = a.scores[row_at];
    if (score == none || (a.finished != nullptr && a.finished[row_at] != 0)) return;
    const T *row = logits + row_at * ld;

    u32x4 r[R];
    if (from + PART <= a.vocab) {
#pragma unroll
        for (int j = 0; j < R; ++j)
            r[j] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4_any *>(row + from + (int64_t)(j * kScanThreads + tid) * VEC));
    } else if (a.vocab >= VEC) {
        // the last part: what ends behind the row is loaded from its end, and shifted
        // into place before -infinity
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int64_t c = from + (int64_t)(j * kScanThreads + tid) * VEC;
            r[j] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4_any *>(row + (c < a.vocab - VEC ? c : a.vocab - VEC)));
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            __builtin_amdgcn_sched_barrier(0);
            const int64_t back = from + (int64_t)(j * kScanThreads + tid + 1) * VEC - a.vocab;
            if (back <= 0) continue;
            r[j] = shift_down<T>(r[j], back < VEC ? (int)back : 0);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (i + back >= VEC) r[j] = with_element<T>(r[j], i, none);
        }
        __builtin_amdgcn_sched_barrier(0);
    } else {
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                r[j] = with_element<T>(r[j], i, j == 0 && tid == 0 && i < a.vocab ? (float)row[i] : none);
    }
    float most[R], of_lane = none;
#pragma unroll
    for (int j = 0; j < R; ++j) {
        most[j] = element<T>(r[j], 0);
#pragma unroll
        for (int i = 1; i < VEC; ++i) most[j] = __builtin_fmaxf(most[j], element<T>(r[j], i));
        of_lane = __builtin_fmaxf(of_lane, most[j]);
    }
    maxima[wave][lane] = key_of(of_lane);
    if (tid == 0) listed = 0, queued = 0;
    __syncthreads();
    if (wave == 0) {
        uint32_t m = 0u;
#pragma unroll
        for (int w = 0; w < kScanWaves; ++w) m = maxima[w][lane] > m ? maxima[w][lane] : m;
        // the upper half of the count-th largest key, bit by bit
        uint32_t key = 0u;
#pragma unroll
        for (int bit = 15; bit >= 0; --bit) {
            const uint32_t trial = key | 1u << bit;
            if (__builtin_popcountll(__builtin_amdgcn_ballot_w64(m >> 16 >= trial)) >= a.count) key = trial;
        }
        const uint32_t top = team_max<kWave>(m);
        if (lane == 0) bound = key == 0u ? 1u : key << 16, largest = top;
    }
    __syncthreads();
    // (the logits that were taken apart are not kept: registers are better used by more
    // waves)
    auto forget = [&] {
#pragma unroll
        for (int j = 0; j < R; ++j) asm("" : "+v"(r[j]));
    };
    forget();
    const uint32_t least_key = bound;
    const float least = least_key == 1u ? -3.402823466e38f : value_of(least_key);
    const float top = value_of(largest);

    if constexpr (SUM) {
        double sum = 0.0;
        auto add = [&](auto &&exponent) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                u32x4 v = r[j];
                asm("" : "+v"(v));
                float e[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) e[i] = __builtin_amdgcn_exp2f(exponent(element<T>(v, i)));
#pragma unroll
                for (int n = VEC / 2; n > 0; n /= 2)
#pragma unroll
                    for (int i = 0; i < n; ++i) e[i] += e[i + n];
                sum += (double)e[0];
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (__builtin_fabsf(top) < kOneProduct) {
            const float base = -(top * kLog2e);
            add([&](float l) { return __builtin_fmaf(l, kLog2e, base); });
        } else {  // large ones, infinities, nothing at all; NaN shows
            add([&](float l) { return l == none ? none : (l - top) * kLog2e; });
        }
        sum = team_sum64<kWave>(sum);
        if (lane == 0) sums[wave] = sum;
        forget();
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const bool has = most[j] >= least;
        const uint64_t those = __builtin_amdgcn_ballot_w64(has);
        if (those == 0ull) continue;
        int at = 0;
        if (lane == 0) at = atomicAdd(&queued, __builtin_popcountll(those));
        at = __builtin_amdgcn_readfirstlane(at) + __builtin_popcountll(those & ((1ull << lane) - 1));
        if (has && at < kQueued) {
            held_all.queue.vector[at] = r[j];
            held_all.queue.token[at] = (uint32_t)from + (uint32_t)(j * kScanThreads + tid) * VEC;
        }
    }
    __syncthreads();
    const int vectors = queued;
    if (vectors <= kQueued)
        for (int at = tid; at < vectors * VEC; at += kScanThreads) {
            constexpr int kPerWord = 4 / (int)sizeof(T);
            const uint32_t word = held_all.queue.vector[at / VEC][at % VEC / kPerWord];
            const u32x4 v = {word, 0u, 0u, 0u};
            const float l = kPerWord == 2 && at % 2 ? element<T>(v, 1 % VEC) : element<T>(v, 0);
            if (l >= least) {
                const int to = atomicAdd(&listed, 1);
                if (to < kListed) list[to] = candidate_of(l, held_all.queue.token[at / VEC] + (uint32_t)(at % VEC));
            }
        }
    __syncthreads();
    int n = listed;
    if (vectors > kQueued || n > kListed) {
        forget();
        uint64_t *held = held_all.of_wave[wave];
        uint64_t above = 0ull;
        n = 0;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const uint32_t token = (uint32_t)from + (uint32_t)(j * kScanThreads + tid) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float l = element<T>(r[j], i);
                const uint64_t c = candidate_of(l, token + i);
                bool takes = l >= least && c > above;
                uint64_t all = __builtin_amdgcn_ballot_w64(takes);
                if (all == 0ull) continue;
                if (n + __builtin_popcountll(all) > kHeld) {
                    n = keep_best(held, n, a.count, lane);
                    if (n == a.count) above = held[n - 1];
                    takes = takes && c > above;
                    all = __builtin_amdgcn_ballot_w64(takes);
                }
                if (takes) held[n + __builtin_popcountll(all & ((1ull << lane) - 1))] = c;
                n += __builtin_popcountll(all);
            }
        }
        n = keep_best(held, n, a.count, lane);
        if (lane < a.count) list[wave * a.count + lane] = lane < n ? held[lane] : 0ull;
        n = kScanWaves * a.count;
        __syncthreads();
    }
    // each candidate's place, by counting those that are better
    uint64_t *best = a.best + job * a.count;
    if (tid < n) {
        const uint64_t mine = list[tid];
        int before = 0;
        for (int i = 0; i < n; ++i) before += list[i] > mine;
        if (mine != 0ull && before < a.count) best[before] = mine;
    }
    if (n < a.count && tid >= n && tid < a.count) best[tid] = 0ull;
    if constexpr (SUM)
        if (tid == 0) {
            double sum = 0.0;
            for (int w = 0; w < kScanWaves; ++w) sum += sums[w];
            const double base = (double)-(top * kLog2e);
            const double of_fma = (double)top * kLog2eLess - base * kLn2;
            a.of_part[job] = Part{sum, __builtin_fabsf(top) < kOneProduct ? of_fma : (double)top};
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
    int beams, parts, count, end_id;
    uint8_t normalize, wide_ids, token_bits;  // bits that hold any token
};

constexpr int kJoinThreads = 1024, kJoinWaves = kJoinThreads / kWave;
constexpr int kJoinHeld = 2;                          // candidates a thread holds
constexpr int kJoinBlock = kJoinThreads * kJoinHeld;  // and the workgroup
constexpr int kRankLanes = 16;                        // lanes that rank one together
constexpr int kRanked = kJoinThreads / kRankLanes;

// A continuation: its total's order key (float64), and by what equal totals are told
// apart, larger being better: the beam (the lowest first), then the order key of its
// logit, which a total may have swallowed, then the token (the lowest first).  Beams
// times tokens are below 2^31, so that the bits of both are 32 at most.
struct Total {
    uint64_t key, place;  // 0, 0: none
};

__device__ __forceinline__ bool better(const Total &a, const Total &b)
{
    return a.key > b.key || (a.key == b.key && a.place > b.place);
}

__device__ __forceinline__ uint64_t place_of(const Join &a, int beam, uint64_t candidate)
{
    const uint64_t before_token = (uint64_t)(uint32_t)(a.beams - 1 - beam) << 32 | candidate >> 32;
    return before_token << a.token_bits | __builtin_amdgcn_ubfe((uint32_t)candidate, 0, a.token_bits);
}

// Totals in LDS, and how many of the first n are better than the i-th: for the 16 lanes
// that ask for the same i.
template <int SIZE>
struct Totals {
    uint64_t key[SIZE], place[SIZE];
    __device__ __forceinline__ Total at(int i) const { return {key[i], place[i]}; }
    __device__ __forceinline__ void set(int i, const Total &t) { key[i] = t.key, place[i] = t.place; }
    __device__ __forceinline__ int before(int i, int n) const
    {
        const Total mine = at(i);
        uint32_t b = 0;
        for (int o = (int)threadIdx.x % kRankLanes; o < n; o += kRankLanes) b += better(at(o), mine);
        return (int)team_reduce<kRankLanes>(b, [](uint32_t x, uint32_t y) { return x + y; });
    }
};

// One workgroup per search: the beams' log sums from their parts; then the candidates of
// all parts at once, a few a thread, those that do not reach the `count`-th largest of 64
// maxima left out, the others ranked by counting.  Bound by latency: 5 us for 4 beams of
// 32,000 logits, 6 for 64 searches of 8 beams of 131,072 (1,024 candidates each); with 512
// threads half a microsecond more, with 256 1.5.  For 32 of beams of like scores 23, 48 17,
// 62 28, 63 84, 64 163: more candidates reach a bound of 64 maxima, the more where `count`
// divides 64 and so each of the 64 is over places of one rank.  Ranking every list's best first, then
// the lists' next places in rounds, took 17 to 33.
__global__ __launch_bounds__(kJoinThreads) void beam_join_kernel(Join a, int batch)
{
    // (a thread's best are looked at for the bound, before what reaches it is taken)
    __shared__ union {
        Totals<kJoinThreads> of_thread;
        Totals<kJoinBlock + kMaxBeams> taken;
    } all_totals;
    auto &of_thread = all_totals.of_thread;
    auto &taken = all_totals.taken;
    __shared__ Totals<kWave> maxima;
    __shared__ Totals<kMaxContinuations> kept;
    __shared__ double norm[kMaxBeams];  // of each beam: what its logits are less
    __shared__ float score[kMaxBeams];  // -infinity: takes no part
    __shared__ int taken_count;
    __shared__ Total bound_total;
    const int tid = (int)threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const float none = -__builtin_inff();
    const Total nothing{0ull, 0ull};
    const int lists = a.beams * a.parts;
    const int64_t all = (int64_t)lists * a.count;

    const int64_t b = blockIdx.y * kMaxGridX + blockIdx.x;
    if (b >= batch) return;
    // the first block's candidates are on their way while the sums are formed
    uint64_t c[kJoinHeld];
    auto load = [&](int64_t base) {
#pragma unroll
        for (int i = 0; i < kJoinHeld; ++i) {
            const int64_t at = base + i * kJoinThreads + tid;
            c[i] = at < all ? a.best[b * all + at] : 0ull;
        }
    };
    load(0);
    for (int beam = wave; beam < a.beams; beam += kJoinWaves) {
        const int64_t row = b * a.beams + beam;
        const float s = a.scores[row];
        const bool over = a.finished != nullptr && a.finished[row] != 0;
        double less = 0.0;
        if (a.normalize && s != none && !over) {
            double high = (double)none;
            for (int p = lane; p < a.parts; p += kWave)
                high = __builtin_fmax(high, a.of_part[row * a.parts + p].base);
#pragma unroll
            for (int d = 1; d < kWave; d *= 2) high = __builtin_fmax(high, __shfl_xor(high, d, kWave));
            double sum = 0.0;
            for (int p = lane; p < a.parts; p += kWave) {
                const Part q = a.of_part[row * a.parts + p];
                sum += q.base == (double)none ? q.sum : q.sum * exp(q.base - high);
            }
            less = high + log(team_sum64<kWave>(sum));
        }
        if (lane == 0) norm[beam] = less, score[beam] = over ? none : s;
    }
    int kept_count = 0;
    __syncthreads();

    for (int64_t base = 0; base == 0 || base < all; base += kJoinBlock) {
        if (base > 0) load(base);
        if (tid == 0) taken_count = 0, bound_total = nothing;
        Total t[kJoinHeld + 1];
#pragma unroll
        for (int i = 0; i < kJoinHeld; ++i) {
            const int64_t at = base + i * kJoinThreads + tid;
            t[i] = nothing;
            if (at >= all || (uint32_t)(c[i] >> 32) == 0u) continue;
            // (a part is a thousand tokens or more: there are far fewer candidates than 2^31)
            const int beam = (int)((uint32_t)at / (uint32_t)(a.parts * a.count));
            if (score[beam] == none) continue;  // (what is there was left by another call)
            t[i] = {key_of((double)score[beam] + ((double)logit_of(c[i]) - norm[beam])), place_of(a, beam, c[i])};
        }
        // with the first block finished beams, with later ones the best so far
        t[kJoinHeld] = nothing;
        if (base > 0) {
            if (tid < kept_count) t[kJoinHeld] = kept.at(tid);
        } else if (tid < a.beams && a.finished != nullptr) {
            const int64_t row = b * a.beams + tid;
            const float s = a.scores[row];
            if (a.finished[row] != 0 && s != none)
                t[kJoinHeld] = {key_of((double)s), place_of(a, tid, ~(uint32_t)a.end_id)};
        }
        Total mine = t[0];
#pragma unroll
        for (int i = 1; i <= kJoinHeld; ++i)
            if (better(t[i], mine)) mine = t[i];
        of_thread.set(tid, mine);
        __syncthreads();
        if (tid < kWave) {
            for (int w = 1; w < kJoinWaves; ++w)
                if (better(of_thread.at(w * kWave + tid), mine)) mine = of_thread.at(w * kWave + tid);
            maxima.set(tid, mine);
        }
        __syncthreads();
        {
            // (of fewer than `count` there is none at that place, and all are taken)
            const int i = tid / kRankLanes;
            const int before = maxima.before(i, kWave);
            if (tid % kRankLanes == 0 && before == a.count - 1) bound_total = maxima.at(i);
        }
        __syncthreads();
        const Total bound = bound_total;
#pragma unroll
        for (int i = 0; i <= kJoinHeld; ++i)
            if (t[i].key != 0ull && !better(bound, t[i])) taken.set(atomicAdd(&taken_count, 1), t[i]);
        __syncthreads();
        const int n = taken_count;
        for (int i = tid / kRankLanes; i < n; i += kRanked) {
            const int before = taken.before(i, n);
            if (tid % kRankLanes == 0 && before < a.count) kept.set(before, taken.at(i));
        }
        kept_count = n < a.count ? n : a.count;
        __syncthreads();
    }
    for (int k = tid; k < a.count; k += kJoinThreads) {
        const int64_t at = b * a.count + k;
        const bool there = k < kept_count;
        const uint64_t place = there ? kept.place[k] : 0ull;
        a.out_scores[at] = there ? (float)value_of(kept.key[k]) : none;
        a.parents[at] = there ? a.beams - 1 - (int)(place >> 32 >> a.token_bits) : -1;
        const int token = there ? (int)__builtin_amdgcn_ubfe(~(uint32_t)place, 0, a.token_bits) : -1;
        if (a.wide_ids)
            ((int64_t *)a.tokens)[at] = token;
        else
            ((int32_t *)a.tokens)[at] = token;
    }
}

// ----------------------------------------------------------------- reordering

struct Places {
    int64_t outer_step, batch_step, beam_step, middle_step, row_step;
};

struct Reorder {
    int64_t vecs, tiles;  // whole vectors of a row, and of these the tiles
    int all_rows, rows, middle, batch, beams, count;
    int8_t words, tx_log2;  // words behind a row's vectors
    bool in_place;
};

// What is moved at once, at any address.
struct Vector {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(1)));
};
struct Word4 {
    typedef uint32_t type __attribute__((aligned(1)));
};
struct Word2 {
    typedef uint16_t type __attribute__((aligned(1)));
};
struct Word1 {
    typedef uint8_t type;
};

// Encoding of a wait for the vector memory counter at zero, and for nothing else.
constexpr int kLoadsDone = 0x0F70;

// What a wave does that serves one row: p[i] is the parent of beam i, and takers[i] the
// beams that its state goes to, if i is the first of them; zeroed, the beams without one.
template <int MOST>
struct Moves {
    using Beams = std::conditional_t<(MOST > 32), uint64_t, uint32_t>;  // a bit for each
    int p[MOST];
    Beams takers[MOST], zeroed;
};

// Found by the wave's first lanes, one for a beam: all lanes call it.  (With the beams
// compared pair by pair in scalar registers, 9 of 5 beams, 9 MB, took 7.9 us instead of 4.7.)
template <int MOST>
__device__ __forceinline__ Moves<MOST> wave_moves(const int32_t *parents, int beams, int count, bool in_place)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int parent = lane < count ? parents[lane] : -1;
    const bool named = (uint32_t)parent < (uint32_t)beams;
    using Beams = typename Moves<MOST>::Beams;
    const Beams needed = (Beams)__ballot(named && !(in_place && parent == lane));
    Moves<MOST> m;
    m.zeroed = (Beams)__ballot(lane < count && !named);
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        m.p[i] = __builtin_amdgcn_readlane(parent, i);
        const Beams same = (Beams)__ballot(parent == m.p[i]) & needed;
        m.takers[i] = (same & (0 - same)) == (Beams)1 << i ? same : 0;
    }
    return m;
}

// A lane moves one column, of 16 bytes or (at a row's end) of one word, of all beams of
// a search: it has read what it needs of the old states before it stores the first of
// the new ones, so they may be the same memory.  in and out are the same for the whole
// wave, `at` is the lane's.  Each state that is needed is read once.
template <typename W, int MOST, bool NT>
__device__ __forceinline__ void move_column(const char *in, int64_t in_step, char *out, int64_t out_step, uint32_t at,
                                            const Moves<MOST> &m)
{
    using T = typename W::type;
    T v[MOST];
#pragma unroll
    for (int i = 0; i < MOST; ++i)
        if (m.takers[i] != 0) {
            const T *from = reinterpret_cast<const T *>(in + m.p[i] * in_step + at);
            if constexpr (NT)
                v[i] = __builtin_nontemporal_load(from);
            else
                v[i] = *from;
        }
    // all loads are waited for here: a wait among the stores would be for stores too
    __builtin_amdgcn_s_waitcnt(kLoadsDone);
    auto store = [&](auto beams, T value) {
#pragma unroll 1
        for (; beams != 0; beams &= beams - 1)
            __builtin_nontemporal_store(value, reinterpret_cast<T *>(out + __builtin_ctzll(beams) * out_step + at));
    };
#pragma unroll
    for (int i = 0; i < MOST; ++i) store(m.takers[i], v[i]);
    store(m.zeroed, T{});
}

// The same where a wave serves several rows, whose parents may differ: a lane finds out
// by itself who takes what.
template <typename W, int MOST, bool NT>
__device__ __forceinline__ void move_lane_column(const char *in, int64_t in_step, char *out, int64_t out_step,
                                                 uint32_t at, const int32_t *parents, int beams, int count,
                                                 bool in_place)
{
    using T = typename W::type;
    int p[MOST];  // all of them first: each is a load
#pragma unroll
    for (int j = 0; j < MOST; ++j) p[j] = parents[j < count ? j : 0];
    auto named = [&](int j) { return (uint32_t)p[j] < (uint32_t)beams; };
    auto stays = [&](int j) { return in_place && p[j] == j && named(j); };
    auto needed = [&](int j) { return j < count && named(j) && !stays(j); };
    T v[MOST];
    if constexpr (MOST <= 16) {
        // the first of the beams that have a parent loads it, for all of them
        bool leads[MOST];
#pragma unroll
        for (int j = 0; j < MOST; ++j) {
            leads[j] = needed(j);
#pragma unroll
            for (int i = 0; i < j; ++i) leads[j] = leads[j] && !(leads[i] && p[i] == p[j]);
        }
#pragma unroll
        for (int j = 0; j < MOST; ++j)
            if (leads[j]) {
                const T *from = reinterpret_cast<const T *>(in + p[j] * in_step + at);
                if constexpr (NT)
                    v[j] = __builtin_nontemporal_load(from);
                else
                    v[j] = *from;
            }
        __builtin_amdgcn_s_waitcnt(kLoadsDone);
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            if (!leads[i]) continue;
#pragma unroll
            for (int j = i; j < MOST; ++j)
                if (needed(j) && p[j] == p[i])
                    __builtin_nontemporal_store(v[i], reinterpret_cast<T *>(out + j * out_step + at));
        }
    } else {
        // (a beam whose state is not needed loads another's again, or the first, which is
        // always there: what is loaded again comes from the caches)
        static_assert(!NT, "loads that the caches answer do not go past them");
        int spare = 0;
#pragma unroll
        for (int j = MOST - 1; j >= 0; --j) spare = needed(j) ? p[j] : spare;
#pragma unroll
        for (int j = 0; j < MOST; ++j)
            v[j] = *reinterpret_cast<const T *>(in + (needed(j) ? p[j] : spare) * in_step + at);
#pragma unroll
        for (int j = 0; j < MOST; ++j)
            if (needed(j)) __builtin_nontemporal_store(v[j], reinterpret_cast<T *>(out + j * out_step + at));
    }
#pragma unroll
    for (int j = 0; j < MOST; ++j)
        if (j < count && !named(j)) __builtin_nontemporal_store(T{}, reinterpret_cast<T *>(out + j * out_step + at));
}

// WORD: the words that a row's last columns are moved in; MOST: beams whose columns a
// lane holds at once (more of them one after another, not in place); NT: loads past the
// caches.
//
// Bound by HBM: caches of 16 searches of 8 beams, 795 MB read and written in place, in
// 133 us (5.9 TB/s, a copy's rate), of one search of 4 beams (22 MB) in 4.9.  A state that
// several beams take is read once: with a load for each beam, which the caches do not
// answer when it goes past them, 140; 9 beams that take one's 27 MB each in 42 us instead
// of 94.  Stores always go past the caches (154 us without, and 41 instead of 32 for 134
// MB of states).
template <typename WORD, int MOST, bool WAVE_ROW, bool NT>
__global__ __launch_bounds__(kThreads) void reorder_kernel(const char *in, char *out,
                                                           const int32_t *__restrict__ all_parents, Places from,
                                                           Places to, Reorder a)
{
    const int64_t r64 = row_of<WAVE_ROW>(a.tx_log2, (int64_t)blockIdx.z * kMaxGridY + blockIdx.y);
    if (r64 >= a.all_rows) return;
    const uint32_t r = (uint32_t)r64;
    const uint32_t block = r / (uint32_t)a.rows, row = r % (uint32_t)a.rows;
    const uint32_t state = block / (uint32_t)a.middle, middle = block % (uint32_t)a.middle;
    const uint32_t outer = state / (uint32_t)a.batch, b = state % (uint32_t)a.batch;
    const char *src = in + outer * from.outer_step + b * from.batch_step + middle * from.middle_step + row * from.row_step;
    char *dst = out + outer * to.outer_step + b * to.batch_step + middle * to.middle_step + row * to.row_step;
    const int32_t *parents = all_parents + (int64_t)b * a.count;
    // tiles of vectors, and behind them one of the words that end a row
    const uint32_t lane = threadIdx.x & ((1u << a.tx_log2) - 1);
#pragma unroll 1
    for (int64_t x = blockIdx.x; x < a.tiles + (a.words > 0); x += kMaxGridX) {
#pragma unroll 1
        for (int j = 0; j < a.count; j += MOST) {
            const int most = a.count - j < MOST ? a.count - j : MOST;
            auto move = [&](auto word, int64_t base, uint32_t at, bool mine) {
                using W = decltype(word);
                const char *in_at = src + base;
                char *out_at = dst + base + j * to.beam_step;
                if constexpr (WAVE_ROW) {
                    const Moves<MOST> m = wave_moves<MOST>(parents + j, a.beams, most, a.in_place);
                    if (mine) move_column<W, MOST, NT>(in_at, from.beam_step, out_at, to.beam_step, at, m);
                } else if (mine) {
                    move_lane_column<W, MOST, NT>(in_at, from.beam_step, out_at, to.beam_step, at, parents + j,
                                                  a.beams, most, a.in_place);
                }
            };
            if (x < a.tiles)
                move(Vector{}, x << a.tx_log2 << 4, lane * 16, (x << a.tx_log2) + lane < a.vecs);
            else
                move(WORD{}, a.vecs * 16, lane * (uint32_t)sizeof(typename WORD::type), lane < (uint32_t)a.words);
        }
    }
}

}  // namespace lrs_choose
