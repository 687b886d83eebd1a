// route_kernels.hpp -- gfx950 (CDNA4, wave64) kernels of a router's choice of experts
// and its gradient (include/lrsort_choose.h).
//
// A team of 8 to 64 lanes serves a token: its logits are loaded once, 16 bytes a
// lane at a time, and stay in registers as order keys while the best are taken from
// them one by one.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "choose_common.hpp"

namespace lrs_choose {

constexpr int kTeamThreads = 128;  // two waves, a token per team
constexpr int kMaxSlots = 64, kMaxGroups = 64;

// -------------------------------------------------------------------- scores

// exp(l) / (1 + exp(l)), and with `low` >= min(l, 0): the same times exp(-low), so that
// the weights of a token whose scores are all below the smallest number keep their
// proportions.
__device__ __forceinline__ float sigmoid_above(float l, float low)
{
    return expf(__builtin_fminf(l, 0.0f) - low) / (1.0f + expf(-__builtin_fabsf(l)));
}

template <typename T>
__device__ __forceinline__ float load_logit(const T *row, int e)
{
    return (float)row[e];
}

struct Route {
    const float *bias;
    void *ids, *weights;
    float scale;
    int tokens;
    int16_t experts, size, groups, kept;  // size: of a group
    uint8_t slots, sigmoid, top2, normalize, wide_ids, weight_type;  // sigmoid: 2 without a bias
    uint8_t lane_groups, lane_groups_log2;  // a group is this many lanes' vectors; 0: it is no such number
};

// A token's list of the chosen, in LDS.
struct Chosen {
    int32_t expert;  // -1: none
    uint32_t key;
};

// exp(x) in float64 for any x but NaN: 2^n exp(r) with n the nearest integer to x log2(e)
// and |r| <= ln(2) / 2, by Taylor's series up to r^13 / 13! (the next term is below
// 2^-57).
__device__ __forceinline__ double exp64(double x)
{
    x = __builtin_fmin(__builtin_fmax(x, -745.0), 709.0);
    const double n = __builtin_rint(x * 1.44269504088896340736);
    // ln(2) in two parts, the first with zeros at its end
    double r = __builtin_fma(n, -0x1.62e42fefap-1, x);
    r = __builtin_fma(n, -0x1.cf79abc9e3b39p-40, r);
    double y = 1.0 / 6227020800.0;
    constexpr double terms[] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0,
                                1.0 / 5040.0,      1.0 / 720.0,      1.0 / 120.0,     1.0 / 24.0,     1.0 / 6.0,
                                0.5,               1.0,              1.0};
#pragma unroll
    for (int i = 0; i < 13; ++i) y = __builtin_fma(y, r, terms[i]);
    return __builtin_ldexp(y, (int)n);
}

// What an expert of logit l is compared by, in float64, as an order key.  By sums: its
// score, for the softmax with the maximum and the sum of its token, and its bias; the
// logit otherwise.
template <bool SUMS>
__device__ __forceinline__ uint64_t choice64(const Route &a, float l, float bias, float top, double sum)
{
    if (l == -__builtin_inff()) return 0ull;
    if constexpr (!SUMS) return key_of((double)l);
    if (bias == -__builtin_inff()) return 0ull;
    double s;
    if (a.sigmoid)
        s = l != l ? (double)l : 1.0 / (1.0 + exp64(-(double)l));
    else
        s = sum != sum ? sum : exp64((double)l - (double)top) / sum;
    return key_of(s + (double)bias);
}

// Whether experts of the kept groups are compared by their logits: a sigmoid rises with
// its logit also where float64 holds one number for both (1 from 37 on).  With a bias
// their sums in float64 decide, and such sums are equal.
template <bool SUMS>
__device__ __forceinline__ bool by_logits(const Route &a)
{
    return SUMS && a.sigmoid == 2;
}

// The softmax's sum in float64, from memory.
template <typename T, int L, int V>
__device__ __forceinline__ double sum64(const T *row, const Route &a, int lane, float top)
{
    if (a.sigmoid) return 1.0;
    double sum = 0.0;
#pragma unroll 4
    for (int i = 0; i < V; ++i) {
        const int e = i * L + lane;
        const float l = e < a.experts ? load_logit(row, e) : -__builtin_inff();
        const double x = (double)l - (double)top;
        sum += l == -__builtin_inff() ? 0.0 : x != x ? x : exp64(x);
    }
    return team_sum64<L>(sum);
}

// A token's scores in float64 as order keys, from memory to LDS (cells: experts, then
// groups, whose scores follow where there is a choice among them).
template <typename T, int L, int V, bool SUMS>
__device__ __forceinline__ void scores_in_64(const T *row, const Route &a, int lane, float top, uint64_t *cells)
{
    const double sum = SUMS ? sum64<T, L, V>(row, a, lane, top) : 1.0;
#pragma unroll 4
    for (int i = 0; i < V; ++i) {
        const int e = i * L + lane;
        if (e < a.experts)
            cells[e] = choice64<SUMS>(a, load_logit(row, e), SUMS && a.bias != nullptr ? a.bias[e] : 0.0f, top, sum);
    }
    wave_sync();
    if (a.kept == a.groups) return;
    for (int g = lane; g < a.groups; g += L) {
        uint64_t first = 0, second = 0;
#pragma unroll 4
        for (int i = 0; i < a.size; ++i) {
            const uint64_t k = cells[g * a.size + i];
            second = k > first ? first : k > second ? k : second;
            first = k > first ? k : first;
        }
        cells[a.experts + g] = a.top2 && second != 0 ? key_of(value_of(first) + value_of(second)) : first;
    }
    wave_sync();
}

// Groups that are better than group g: key[0..groups) their scores.
template <typename K>
__device__ __forceinline__ int groups_before(const K *key, int groups, K mine, int g)
{
    int n = 0;
    for (int o = 0; o < groups; ++o) n += key[o] > mine || (key[o] == mine && o < g);
    return n;
}

// The choice by float64 throughout, for the token whose scores are too close to one
// another in float32, or hold NaN or infinity.
template <typename T, int L, int V, bool SUMS>
__device__ void choose_in_64(const T *row, const Route &a, int lane, float top, uint64_t *cells, Chosen *list)
{
    scores_in_64<T, L, V, SUMS>(row, a, lane, top, cells);
    if (a.kept < a.groups) {
        const uint64_t *of_group = cells + a.experts;
        for (int g = lane; g < a.groups; g += L)
            if (groups_before(of_group, a.groups, of_group[g], g) >= a.kept)
                for (int i = 0; i < a.size; ++i) cells[g * a.size + i] = 0;
        wave_sync();
    }
    if (by_logits<SUMS>(a)) {
#pragma unroll 4
        for (int i = 0; i < V; ++i) {
            const int e = i * L + lane;
            if (e < a.experts && cells[e] != 0) cells[e] = key_of((double)load_logit(row, e));
        }
    }
    for (int k = 0; k < a.slots; ++k) {
        uint64_t best = 0;
        uint32_t at = ~0u;
#pragma unroll 4
        for (int i = 0; i < V; ++i) {
            const int e = i * L + lane;
            const uint64_t c = e < a.experts ? cells[e] : 0ull;
            at = c > best ? (uint32_t)e : at;
            best = c > best ? c : best;
        }
        const uint64_t of_all = team_max64<L>(best);
        at = team_min<L>(best == of_all ? at : ~0u);
        if (of_all != 0 && (int)at % L == lane) cells[at] = 0;
        if (lane == 0) list[k] = {of_all != 0 ? (int)at : -1, 0u};
        wave_sync();
    }
}

// The first `n` of the list, which are the best n of their token, in the order of
// float64.
template <typename T, int L, bool SUMS>
__device__ __forceinline__ void order_in_64(const T *row, const Route &a, int lane, float top, double sum,
                                            uint64_t *cells, Chosen *list, int n)
{
    for (int k = lane; k < n; k += L) {
        const int e = list[k].expert;
        const float l = e < 0 ? -__builtin_inff() : load_logit(row, e);
        const float bias = SUMS && a.bias != nullptr && e >= 0 ? a.bias[e] : 0.0f;
        cells[k] = by_logits<SUMS>(a) ? key_of((double)l) : choice64<SUMS>(a, l, bias, top, sum);
    }
    wave_sync();
    // (a lane has one or a few of them: it reads them all before any is replaced)
    int expert[kMaxSlots / 8 + 1], place[kMaxSlots / 8 + 1];
#pragma unroll
    for (int i = 0; i < kMaxSlots / L + 1; ++i) {
        const int k = i * L + lane;
        if (k >= n) continue;
        expert[i] = list[k].expert;
        place[i] = 0;
        const uint64_t mine = cells[k];
        for (int o = 0; o < n; ++o)
            place[i] += cells[o] > mine || (cells[o] == mine && (uint32_t)list[o].expert < (uint32_t)expert[i]) ||
                        (mine == 0ull && cells[o] == 0ull && o < k);
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < kMaxSlots / L + 1; ++i)
        if (i * L + lane < n) list[place[i]].expert = expert[i];
    wave_sync();
}

// The bits of an order key that follow from a 16-bit logit's others: zeros, or ones where
// it is negative.
constexpr uint32_t kFree = 0x1FFFu;

__device__ __forceinline__ float logit_of_key(uint32_t k)
{
    return value_of(k & 0x80000000u ? k & ~kFree : k | kFree);
}

// Sorts a lane's keys, the largest first, by Batcher's odd-even merges.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&k)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j <= N - 1 - q; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t x = k[i + j], y = k[i + j + q];
                        k[i + j] = x > y ? x : y;
                        k[i + j + q] = x > y ? y : x;
                    }
}

// The choice of `slots` experts per token, and their weights.  Team of L lanes, V logits a
// lane.  SUMS: the choice is by sums (a bias, or groups by their two best) and not by the
// logits themselves.
//
// Each lane sorts its keys; then the best of the lanes' first keys is taken off, one after
// another.  So that a key tells its expert, its last bits are replaced: the 13 that a
// 16-bit logit leaves free by the expert's id, which changes no order but that of equal
// ones, or the last few bits of float32 by the place within the lane.  These then decide nothing: where two
// neighbours of the list are closer than that and the sums' rounding, they are ordered by
// float64, and where the end of the list is not certain either, the choice is made by
// float64 throughout.
//
// Bound by instructions: 16,384 tokens of 256 float32 logits by sigmoid, bias and groups
// of two best in 16.7 us, some 400 vector instructions a token (scores 64, groups 75,
// sorting and packing 45, taking ten off 70, weights 60; the bytes would take 2.7 us), of
// which 2 us are the few waves that go on in float64; without bias and groups 10.3, of
// bf16 7.5.  4 tokens of 128 experts take 3.7, most of it a launch's own time.  Sixteen
// lanes a token up to 256 experts (with 32 it takes 18.9 and 11.7 us), 32 up to 512 (29
// us; 36 with 16).  Taking off the best by a search through all of a lane's keys instead
// of from sorted ones took 24 us; the choice of a close token wholly in float64 16 more.
//
// What float64 costs where most tokens need it (the same sizes, calls in a graph, one
// group / kept by the best / by the two best; 14 / 16 / 18 us by sigmoid with a bias where
// few do, 17 / 19 / 25 by softmax).  `error` is absolute, so scores near zero are all close:
// softmax of logits of standard deviation 4 with a bias 41 / 50 / 48, of 20 46 / 64 / 60;
// sigmoids around exp(-20) with a bias that tells them apart 14 / 17 / 40, without one by
// the two best 57; all logits and biases equal 32 / 53 / 54 by sigmoid, 39 / 65 / 66 by
// softmax.  A bias of -1e30 that leaves one expert of each group makes all groups by two
// close: 28 by sigmoid, 34 by softmax, where -infinity takes 14 and 13.
template <typename T, int L, int V, bool SUMS>
__global__ __launch_bounds__(kTeamThreads) void route_kernel(const T *__restrict__ logits, int64_t ld, Route a,
                                                             int team_bytes)
{
    extern __shared__ uint64_t lds[];
    constexpr int VEC = kVec<T>;
    static_assert(V % VEC == 0, "whole vectors");
    constexpr int kTeams = kTeamThreads / L, J = V / VEC;
    constexpr bool HALF = !SUMS && sizeof(T) == 2;
    const int lane = (int)threadIdx.x % L, team = (int)threadIdx.x / L;
    Chosen *list = reinterpret_cast<Chosen *>(reinterpret_cast<char *>(lds) + team * team_bytes);
    uint64_t *cells64 = reinterpret_cast<uint64_t *>(list + a.slots + 2);
    uint32_t *cells = reinterpret_cast<uint32_t *>(cells64);
    const float none = -__builtin_inff();

    const int64_t t = (blockIdx.y * kMaxGridX + blockIdx.x) * kTeams + team;
    const bool live = t < a.tokens;
    const T *row = logits + (live ? t : 0) * ld;
    u32x4 raw[J];
#pragma unroll
    for (int j = 0; j < J; ++j) raw[j] = issue<T>(row, col_of<T>(a.experts, (int64_t)(j * L + lane) * VEC));
    for (int k = lane; k < a.slots + 2; k += L) list[k] = {-1, 0u};
    // element i of a lane is expert (i / VEC * L + lane) * VEC + i % VEC
    float l[V];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const Col col = col_of<T>(a.experts, (int64_t)(j * L + lane) * VEC);
        const u32x4 r = settle<T>(raw[j], col);
#pragma unroll
        for (int i = 0; i < VEC; ++i) l[j * VEC + i] = live && i < col.valid ? element<T>(r, i) : none;
    }

    // the softmax's maximum and sum over all experts, where they are needed; the
    // exponent's product in two parts, so that its rounding is all that is lost
    float top = 0.0f, sum = 1.0f;
    if (!a.sigmoid && (SUMS || !a.normalize)) {
        top = none;
#pragma unroll
        for (int i = 0; i < V; ++i) top = __builtin_fmaxf(top, l[i]);
        top = team_maxf<L>(top);
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float d = l[i] - top;
            const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(d, 1.44269504f, d * 1.92596303e-8f));
            sum += l[i] == none ? 0.0f : e;
        }
        sum = team_sum<L>(sum);
        if (sum == 0.0f) sum = 1.0f;
    }

    // What is compared, as an order key: the logits, or the scores with their bias, a pair
    // of them off by at most 2 `error` but for the rounding of the sums with the bias, which
    // is counted where they are compared.  In units of 2^-24: an exponential is off by 2.3 |d|
    // + 2 of itself (the difference, its product with the rounded log2(e), the exponential).
    // A sigmoid: 1.3 |l| + 2 (no difference) times s (1 - s), below 0.8, an addition and a
    // reciprocal, together less than 4.  A softmax's score, of 1 / sum at most: 2.1 and a
    // product, less than 4 / sum; and the error of 1 / sum, which is the same for all scores
    // of a token and so counts once in their difference: V + 6 additions, a quotient, and the
    // terms' own 2 |d| + 2 with |d| their mean, weighted, 5.1 at most for 2,048 experts: less
    // than (V + 20) / sum.  Together 8 + V + 20, within 2 (V + 16).
    float error = 0.0f;
    bool close = false;  // too close for float32
    uint32_t key[V];
    if constexpr (SUMS) {
        const float each = 1.0f / sum;
        error = a.sigmoid ? 4 * 0x1p-24f : (V + 16) * 0x1p-24f * each;
        const float shift = a.sigmoid ? 0.0f : top;
        const float by = a.sigmoid ? -1.44269504f : 1.44269504f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float b[VEC];
            if (a.bias != nullptr) {
                // (float32: one or two vectors for one of the logits)
#pragma unroll
                for (int h = 0; h < VEC / 4; ++h) {
                    const Col col = col_of<float>(a.experts, (int64_t)(j * L + lane) * VEC + 4 * h);
                    const u32x4 r = load_col<float>(a.bias, col);
#pragma unroll
                    for (int i = 0; i < 4; ++i) b[4 * h + i] = element<float>(r, i);
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) b[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float x = l[j * VEC + i], e = __builtin_amdgcn_exp2f((x - shift) * by);
                float c = (a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + e) : e * each) + b[i];
                c = x == none ? none : c;
                close |= __builtin_isfpclass(c, 0x203);  // NaN or +infinity
                const uint32_t bits = __builtin_bit_cast(uint32_t, c + 0.0f);
                key[j * VEC + i] = c == none ? 0u : bits ^ ((uint32_t)((int32_t)bits >> 31) | 0x80000000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = key_of(l[i]);
    }

    if (a.kept < a.groups) {
        uint32_t *of_group = cells + a.experts;
        float magnitude = 0.0f;  // of what is added up: its rounding counts, not the sum's
        auto score = [&](uint32_t first, uint32_t second) {
            if (!a.top2 || second == 0u) return first;
            const float x = value_of(first), y = value_of(second);
            magnitude = __builtin_fmaxf(magnitude, __builtin_fabsf(x) + __builtin_fabsf(y));
            return key_of(x + y);
        };
        if (a.lane_groups != 0) {
            // a group's vectors lie in neighbouring lanes
#pragma unroll
            for (int j = 0; j < J; ++j) {
                uint32_t first = key[j * VEC], second = 0u;
                auto join = [&](uint32_t f, uint32_t s) {
                    const uint32_t low = f < first ? f : first;
                    second = s > second ? s : second;
                    second = low > second ? low : second;
                    first = f > first ? f : first;
                };
#pragma unroll
                for (int i = 1; i < VEC; ++i) join(key[j * VEC + i], 0u);
                if (a.lane_groups > 1) join(dpp<0xB1>(first), dpp<0xB1>(second));
                if (a.lane_groups > 2) join(dpp<0x4E>(first), dpp<0x4E>(second));
                if (a.lane_groups > 4) join(dpp<0x141>(first), dpp<0x141>(second));
                if (a.lane_groups > 8) join(dpp<0x140>(first), dpp<0x140>(second));
                const uint32_t mine = score(first, second);
                const int g = (j * L + lane) >> a.lane_groups_log2;
                if (g < a.groups && (lane & (a.lane_groups - 1)) == 0) of_group[g] = mine;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = (i / VEC * L + lane) * VEC + i % VEC;
                if (e < a.experts) cells[e] = key[i];
            }
            wave_sync();
            for (int g = lane; g < a.groups; g += L) {
                uint32_t first = 0u, second = 0u;
                int i = lane % a.size;  // lanes begin at different banks
                for (int n = 0; n < a.size; ++n) {
                    const uint32_t k = cells[g * a.size + i];
                    second = k > first ? first : k > second ? k : second;
                    first = k > first ? k : first;
                    i = i + 1 == a.size ? 0 : i + 1;
                }
                of_group[g] = score(first, second);
            }
        }
        wave_sync();
        // each group's place; and the least of the kept, the most of the others
        uint32_t least = ~0u, most = 0u;
        uint64_t stays = 0;
        for (int g = lane; g < a.groups; g += L) {
            const uint32_t mine = of_group[g];
            const bool s = groups_before(of_group, a.groups, mine, g) < a.kept;
            least = s && mine < least ? mine : least;
            most = !s && mine > most ? mine : most;
            stays |= (uint64_t)s << g;
        }
        if constexpr (SUMS) {
            const float x = value_of(team_min<L>(least)), y = value_of(team_max<L>(most));
            const float size = __builtin_fmaxf(team_maxf<L>(magnitude), __builtin_fabsf(x) + __builtin_fabsf(y));
            const bool near = y != none && !(x - y > 4 * error + size * 0x1p-22f);
            if (near && live) {  // (the same for the whole team)
                wave_sync();
                scores_in_64<T, L, V, SUMS>(row, a, lane, top, cells64);
                const uint64_t *of_group64 = cells64 + a.experts;
                stays = 0;
                for (int g = lane; g < a.groups; g += L)
                    stays |= (uint64_t)(groups_before(of_group64, a.groups, of_group64[g], g) < a.kept) << g;
            }
        }
        const uint32_t low = team_or<L>((uint32_t)stays), high = team_or<L>((uint32_t)(stays >> 32));
        stays = (uint64_t)high << 32 | low;
        if (a.lane_groups != 0) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const bool s = stays >> (((j * L + lane) >> a.lane_groups_log2) & 63) & 1;
#pragma unroll
                for (int i = 0; i < VEC; ++i) key[j * VEC + i] = s ? key[j * VEC + i] : 0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = (i / VEC * L + lane) * VEC + i % VEC;
                key[i] = stays >> (e / a.size & 63) & 1 ? key[i] : 0u;
            }
        }
    }

    // Keys that tell their expert, or their place.  (float32 logits that came from 16 bits
    // are told by their last bits, the whole wave's: 16,384 tokens of 256 in 8.3 us instead
    // of 22.4, most of them having equal logits among their best; 10.3 instead of 9.5 where
    // they did not.)
    bool exact = HALF;
    if constexpr (!HALF && !SUMS) {
        uint32_t used = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i) used |= __builtin_bit_cast(uint32_t, l[i]);
        exact = __builtin_amdgcn_ballot_w64((used & kFree) != 0u) == 0ull;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t e = kFree - (uint32_t)((i / VEC * L + lane) * VEC + i % VEC);
        key[i] = key[i] == 0u ? 0u
                 : exact      ? (key[i] & ~kFree) | e
                              : (key[i] & ~(uint32_t)(V - 1)) | (uint32_t)(V - 1 - i);
    }
    sort_down(key);
    // the best, one after another; where their order is not yet certain two more, to see
    // how far those behind the list are
    const int rounds = a.slots + (exact ? 0 : 2);
    constexpr int kShallow = V < 10 ? V : 10;  // a lane gives up no more in so many rounds
    const bool deep = rounds > kShallow;
    for (int k = 0; k < rounds; ++k) {
        const uint32_t best = team_max<L>(key[0]);
        bool own = key[0] == best && best != 0u;
        if (!exact) {
            // of several lanes that have it the lowest (more owners than teams that have any)
            const uint64_t those = __builtin_amdgcn_ballot_w64(own);
            constexpr uint64_t kFirst = L == 64   ? 1ull
                                        : L == 32 ? 0x0000000100000001ull
                                        : L == 16 ? 0x0001000100010001ull
                                                  : 0x0101010101010101ull;
            if (__builtin_popcountll(those) != __builtin_popcountll(__builtin_amdgcn_ballot_w64(best != 0u) & kFirst)) {
                const uint64_t mine = those >> (threadIdx.x % kWave / L * L);
                own = own && (mine & ((1ull << lane) - 1)) == 0ull;
            }
        }
        if (own) list[k] = {lane, best};
        auto shift = [&](int from, int to) {
#pragma unroll
            for (int i = from; i < to; ++i) {
                const uint32_t here = key[i], next = i + 1 < V ? key[i + 1 < V ? i + 1 : 0] : 0u;
                key[i] = own ? next : here;
            }
        };
        shift(0, kShallow);
        if (V > kShallow && deep) shift(kShallow, V);
    }
    wave_sync();
    // from the lanes and their keys the experts
    for (int k = lane; k < rounds; k += L) {
        const Chosen c = list[k];
        if (c.expert < 0) continue;
        const int i = V - 1 - (int)(c.key & (V - 1));
        list[k].expert = exact ? (int)(kFree - (c.key & kFree)) : (i / VEC * L + c.expert) * VEC + i % VEC;
    }
    wave_sync();
    if (!exact) {
        bool order = false, end = false;
        for (int k = lane; k <= a.slots; k += L) {
            const uint32_t kx = list[k].key & ~(uint32_t)(V - 1), ky = list[k + 1].key & ~(uint32_t)(V - 1);
            const float x = value_of(kx), y = value_of(ky);
            // (a logit with other bits above those replaced is larger)
            const bool near = ky != 0u && (SUMS ? !(x - y > 2 * error + (__builtin_fabsf(x) + __builtin_fabsf(y)) *
                                                                              ((V + 2) * 0x1p-23f))
                                                : kx == ky);
            order |= near && k < a.slots;
            end |= near && k == a.slots;
        }
        // (a close end matters where the list's last place is close to it too)
        order = team_or<L>(order && live) != 0u;
        end = team_or<L>(end) != 0u;
        close = team_or<L>(close && live) != 0u || (end && order);
        if (close)
            choose_in_64<T, L, V, SUMS>(row, a, lane, top, cells64, list);
        else if (order) {
            double sum = 1.0;
            if constexpr (SUMS)
                if (!a.sigmoid) {
                    // (no NaN is here: it would be close)
                    sum = 0.0;
#pragma unroll
                    for (int i = 0; i < V; ++i) sum += l[i] == none ? 0.0 : exp64((double)l[i] - (double)top);
                    sum = team_sum64<L>(sum);
                }
            order_in_64<T, L, SUMS>(row, a, lane, top, sum, cells64, list, a.slots + 1);
        }
    }

    // weights: of each chosen logit, by the softmax's or the sigmoid's parts
    float high = none;
    for (int k = lane; k < a.slots; k += L) {
        const int e = list[k].expert;
        const float x = e < 0 ? none : HALF ? logit_of_key(list[k].key) : load_logit(row, e);
        list[k].key = __builtin_bit_cast(uint32_t, x);  // from here on the logit
        high = __builtin_fmaxf(high, x);
    }
    float total = 1.0f;
    if (a.normalize) {
        high = team_maxf<L>(high);
        if (a.sigmoid) high = __builtin_fminf(high, 0.0f);
        total = 0.0f;
        for (int k = lane; k < a.slots; k += L)
            if (list[k].expert >= 0) {
                const float x = __builtin_bit_cast(float, list[k].key);
                total += a.sigmoid ? sigmoid_above(x, high) : expf(x - high);
            }
        total = team_sum<L>(total);
        if (SUMS && sum != sum) total = sum;  // a NaN that was not chosen itself
    } else {
        high = a.sigmoid ? 0.0f : top;
        total = sum;
    }
    if (live)
        for (int k = lane; k < a.slots; k += L) {
            const int64_t at = t * a.slots + k;
            const int e = list[k].expert;
            if (a.wide_ids)
                ((int64_t *)a.ids)[at] = e;
            else
                ((int32_t *)a.ids)[at] = e;
            if (a.weights == nullptr) continue;
            const float x = __builtin_bit_cast(float, list[k].key);
            const float w = a.sigmoid ? sigmoid_above(x, high) : expf(x - high);
            store_scalar(a.weights, a.weight_type, at, e < 0 ? 0.0f : a.scale * (w / total));
        }
}

// ------------------------------------------------------------------ gradient

struct RouteGrad {
    const void *ids, *grad_weights;
    float scale;
    int tokens;
    int16_t experts;
    uint8_t slots, sigmoid, normalize, wide_ids, weight_type;
};

struct Share {
    int32_t expert;  // -1: no part
    float by;
};

// A row of gradients is put together in LDS (zeros, and a share at each chosen expert)
// and stored in vectors.  WHOLE: the softmax without normalisation, where every logit
// has its share, p = s * (1 / sum): two roundings, 2^-24 more than a division for each, with
// which the calls below take 11.0 us in a graph instead of 10.6.  Bound by latency, a wave's
// loads, then its stores: 16,384 tokens of 256 float32 logits in 10 us (35 MB, 3.5 TB/s; by
// the bytes 5), 7.6 where the logits of the chosen alone are read.
template <typename T, int L, int V, bool WHOLE>
__global__ __launch_bounds__(kTeamThreads) void route_grad_kernel(const T *logits, int64_t ld, T *grad_logits,
                                                                  int64_t ld_grad, RouteGrad a, int team_bytes)
{
    extern __shared__ uint64_t lds[];
    constexpr int VEC = kVec<T>;
    constexpr int kTeams = kTeamThreads / L;
    const int lane = (int)threadIdx.x % L, team = (int)threadIdx.x / L;
    float *cells = reinterpret_cast<float *>(reinterpret_cast<char *>(lds) + team * team_bytes);
    Share *list = reinterpret_cast<Share *>(cells + L * V);
    float *grads = reinterpret_cast<float *>(list + a.slots);
    const float none = -__builtin_inff();

    const int64_t t = (blockIdx.y * kMaxGridX + blockIdx.x) * kTeams + team;
    const bool live = t < a.tokens;
    const T *row = logits + (live ? t : 0) * ld;
    float s[WHOLE ? V : 1];
    float top = 0.0f, sum = 1.0f;
    if constexpr (WHOLE) {
        u32x4 raw[V / VEC];
#pragma unroll
        for (int j = 0; j < V / VEC; ++j)
            raw[j] = issue<T>(row, col_of<T>(a.experts, (int64_t)(j * L + lane) * VEC));
        top = none;
#pragma unroll
        for (int j = 0; j < V / VEC; ++j) {
            const Col col = col_of<T>(a.experts, (int64_t)(j * L + lane) * VEC);
            const u32x4 r = settle<T>(raw[j], col);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float l = i < col.valid ? element<T>(r, i) : none;
                s[j * VEC + i] = l;
                top = __builtin_fmaxf(top, l);
            }
        }
        top = team_maxf<L>(top);
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float d = s[i] - top;
            const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(d, 1.44269504f, d * 1.92596303e-8f));
            s[i] = s[i] == none ? 0.0f : e;
            sum += s[i];
        }
        sum = team_sum<L>(sum);
        if (sum == 0.0f) sum = 1.0f;
    }
#pragma unroll
    for (int j = 0; j < V / VEC; ++j)
#pragma unroll
        for (int i = 0; i < VEC; i += 4)
            *reinterpret_cast<u32x4 *>(cells + (j * L + lane) * VEC + i) = u32x4{0u, 0u, 0u, 0u};

    // each place's expert, logit and gradient (loaded with the id: what belongs to no
    // expert is not used); then its share
    float high = none;
    for (int k = lane; k < a.slots; k += L) {
        const int64_t at = t * a.slots + k;
        int64_t id = -1;
        if (live) {
            id = a.wide_ids ? ((const int64_t *)a.ids)[at] : ((const int32_t *)a.ids)[at];
            grads[k] = a.scale * load_scalar(a.grad_weights, a.weight_type, at);
        }
        int e = (uint64_t)id < (uint64_t)a.experts ? (int)id : -1;
        const float l = e < 0 ? none : load_logit(row, e);
        if (l == none) e = -1;
        list[k] = {e, l};
        high = __builtin_fmaxf(high, l);
    }
    float total = sum;
    if (a.normalize) {
        high = team_maxf<L>(high);
        if (a.sigmoid) high = __builtin_fminf(high, 0.0f);
        total = 0.0f;
        for (int k = lane; k < a.slots; k += L)
            if (list[k].expert >= 0) total += a.sigmoid ? sigmoid_above(list[k].by, high) : expf(list[k].by - high);
        total = team_sum<L>(total);
    } else {
        high = a.sigmoid ? 0.0f : top;
    }
    float dot = 0.0f;  // of the weights and their gradients
    for (int k = lane; k < a.slots; k += L)
        if (list[k].expert >= 0) {
            const float l = list[k].by, w = (a.sigmoid ? sigmoid_above(l, high) : expf(l - high)) / total;
            dot += w * grads[k];
        }
    dot = team_sum<L>(dot);
    for (int k = lane; k < a.slots; k += L)
        if (list[k].expert >= 0) {
            const float l = list[k].by, w = (a.sigmoid ? sigmoid_above(l, high) : expf(l - high)) / total;
            const float d = w * (a.normalize ? grads[k] - dot : grads[k]);
            list[k].by = a.sigmoid ? d * sigmoid_above(-l, 0.0f) : d;
        }
    wave_sync();
    // an expert's first place writes the sum over all places that name it, in their order
    for (int k = lane; k < a.slots; k += L) {
        const int e = list[k].expert;
        bool first = e >= 0;
        for (int o = 0; o < k; ++o) first &= list[o].expert != e;
        if (!first) continue;
        float d = list[k].by;
        for (int o = k + 1; o < a.slots; ++o) d += list[o].expert == e ? list[o].by : 0.0f;
        cells[e] = d;
    }
    wave_sync();
    if (live) {
        T *out = grad_logits + t * ld_grad;
        const float each = 1.0f / sum;
#pragma unroll
        for (int j = 0; j < V / VEC; ++j) {
            const Col col = col_of<T>(a.experts, (int64_t)(j * L + lane) * VEC);
            float d[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                d[i] = cells[(j * L + lane) * VEC + i];
                if constexpr (WHOLE) {
                    // (a score of zero has no share in a NaN that it did not cause)
                    const float p = s[j * VEC + i] * each;
                    d[i] -= p == 0.0f ? 0.0f : p * dot;
                }
            }
            store_col<T>(out, pack<T>(d), col);
        }
    }
}

}  // namespace lrs_choose
