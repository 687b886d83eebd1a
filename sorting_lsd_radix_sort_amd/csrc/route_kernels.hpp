// route_kernels.hpp -- gfx950 (CDNA4, wave64) kernels of a router's choice of experts
// and its gradient (include/lrsort_choose.h).
//
// A team of 8, 16 or 64 lanes serves a token: its logits are loaded once, 16 bytes a
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
    uint8_t slots, sigmoid, top2, normalize, wide_ids, weight_type;
};

// A token's list of the chosen, in LDS.
struct Chosen {
    int32_t expert;  // -1: none
    uint32_t key;
};

// The choice by float64, for the token whose scores are too close to one another in
// float32: all of its scores again, from memory to LDS (cells: experts, then groups).
template <typename T, int L>
__device__ void choose_in_64(const T *row, const Route &a, int lane, float top, uint64_t *cells, Chosen *list)
{
    double sum = 1.0;
    if (!a.sigmoid) {
        sum = 0.0;
        for (int e = lane; e < a.experts; e += L) {
            const float l = load_logit(row, e);
            sum += l == -__builtin_inff() ? 0.0 : exp((double)l - (double)top);
        }
        sum = team_sum64<L>(sum);
    }
    for (int e = lane; e < a.experts; e += L) {
        const float l = load_logit(row, e), b = a.bias != nullptr ? a.bias[e] : 0.0f;
        const double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top) / sum;
        cells[e] = l == -__builtin_inff() || b == -__builtin_inff() ? 0ull : key_of(s + (double)b);
    }
    wave_sync();
    if (a.kept < a.groups) {
        uint64_t *of_group = cells + a.experts;
        for (int g = lane; g < a.groups; g += L) {
            uint64_t first = 0, second = 0;
            for (int i = 0; i < a.size; ++i) {
                const uint64_t k = cells[g * a.size + i];
                second = k > first ? first : k > second ? k : second;
                first = k > first ? k : first;
            }
            of_group[g] = a.top2 && second != 0 ? key_of(value_of(first) + value_of(second)) : first;
        }
        wave_sync();
        for (int g = lane; g < a.groups; g += L) {
            int before = 0;
            for (int o = 0; o < a.groups; ++o) before += of_group[o] > of_group[g] || (of_group[o] == of_group[g] && o < g);
            if (before >= a.kept)
                for (int i = 0; i < a.size; ++i) cells[g * a.size + i] = 0;
        }
        wave_sync();
    }
    for (int k = 0; k < a.slots; ++k) {
        uint64_t best = 0;
        uint32_t at = ~0u;
        for (int e = lane; e < a.experts; e += L)
            if (cells[e] > best) best = cells[e], at = (uint32_t)e;
        const uint64_t of_all = team_max64<L>(best);
        at = team_min<L>(best == of_all ? at : ~0u);
        if (of_all != 0 && (int)at % L == lane) cells[at] = 0;
        if (lane == 0) list[k] = {of_all != 0 ? (int)at : -1, 0u};
        wave_sync();
    }
}

// The choice of `slots` experts per token, and their weights.  Team of L lanes, V logits a
// lane.  SUMS: the choice is by sums (a bias, or groups by their two best) and not by the
// logits themselves.
template <typename T, int L, int V, bool SUMS>
__global__ __launch_bounds__(kTeamThreads) void route_kernel(const T *__restrict__ logits, int64_t ld, Route a,
                                                             int team_bytes)
{
    extern __shared__ uint64_t lds[];
    constexpr int VEC = kVec<T>;
    static_assert(V % VEC == 0, "whole vectors");
    constexpr int kTeams = kTeamThreads / L;
    const int lane = (int)threadIdx.x % L, team = (int)threadIdx.x / L;
    Chosen *list = reinterpret_cast<Chosen *>(reinterpret_cast<char *>(lds) + team * team_bytes);
    uint64_t *cells64 = reinterpret_cast<uint64_t *>(list + a.slots + 2);
    uint32_t *cells = reinterpret_cast<uint32_t *>(cells64);
    const float none = -__builtin_inff();

    for (int64_t t = (int64_t)blockIdx.x * kTeams + team; t - team < a.tokens; t += kMaxGridX * kTeams) {
        const bool live = t < a.tokens;
        const T *row = logits + (live ? t : 0) * ld;
        u32x4 raw[V / VEC];
#pragma unroll
        for (int j = 0; j < V / VEC; ++j) raw[j] = issue<T>(row, col_of<T>(a.experts, (int64_t)(j * L + lane) * VEC));
        // element i of a lane is expert (i / VEC * L + lane) * VEC + i % VEC
        uint32_t key[V];
#pragma unroll
        for (int j = 0; j < V / VEC; ++j) {
            const Col col = col_of<T>(a.experts, (int64_t)(j * L + lane) * VEC);
            const u32x4 r = settle<T>(raw[j], col);
#pragma unroll
            for (int i = 0; i < VEC; ++i) key[j * VEC + i] = live && i < col.valid ? key_of(element<T>(r, i)) : 0u;
        }
        uint32_t local = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i) local = key[i] > local ? key[i] : local;

        // the softmax's maximum and sum over all experts, where they are needed
        float top = 0.0f, sum = 1.0f;
        if (!a.sigmoid && (SUMS || !a.normalize)) {
            const uint32_t best = team_max<L>(local);
            top = value_of(best);
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += key[i] == 0u ? 0.0f : expf(value_of(key[i]) - top);
            sum = best == 0u ? 1.0f : team_sum<L>(sum);
        }

        // what is compared: the logits, or the scores with their bias, off by at most
        // `error` (counted below) but for the sum's rounding
        float error = 0.0f;
        if constexpr (SUMS) {
            const float each = 1.0f / sum;
            error = a.sigmoid ? 8 * 0x1p-24f : 64 * 0x1p-24f * each;
            local = 0u;
#pragma unroll
            for (int j = 0; j < V / VEC; ++j) {
                const int c = (j * L + lane) * VEC;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    uint32_t &k = key[j * VEC + i];
                    const float l = value_of(k), b = a.bias != nullptr && c + i < a.experts ? a.bias[c + i] : 0.0f;
                    const float s = a.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - top) * each;
                    k = k == 0u || b == none ? 0u : key_of(s + b);
                    local = k > local ? k : local;
                }
            }
        }

        bool close = false;  // too close for float32
        if (a.kept < a.groups) {
            uint32_t *of_group = cells + a.experts;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = (i / VEC * L + lane) * VEC + i % VEC;
                if (e < a.experts) cells[e] = key[i];
            }
            wave_sync();
            float magnitude = 0.0f;  // of what is added up: its rounding counts, not the sum's
            for (int g = lane; g < a.groups; g += L) {
                uint32_t first = 0u, second = 0u;
                int i = lane % a.size;  // lanes begin at different banks
                for (int n = 0; n < a.size; ++n) {
                    const uint32_t k = cells[g * a.size + i];
                    second = k > first ? first : k > second ? k : second;
                    first = k > first ? k : first;
                    i = i + 1 == a.size ? 0 : i + 1;
                }
                const float x = value_of(first), y = a.top2 && second != 0u ? value_of(second) : 0.0f;
                of_group[g] = first == 0u ? 0u : key_of(x + y);
                if (first != 0u) magnitude = __builtin_fmaxf(magnitude, __builtin_fabsf(x) + __builtin_fabsf(y));
            }
            wave_sync();
            uint32_t least = ~0u, most = 0u;  // of the kept, of the others
            for (int g = lane; g < a.groups; g += L) {
                const uint32_t mine = of_group[g];
                int before = 0;
                for (int o = 0; o < a.groups; ++o) before += of_group[o] > mine || (of_group[o] == mine && o < g);
                if (before < a.kept) {
                    least = mine < least ? mine : least;
                } else {
                    most = mine > most ? mine : most;
                    for (int i = 0; i < a.size; ++i) cells[g * a.size + i] = 0u;
                }
            }
            wave_sync();
            if constexpr (SUMS) {
                const float x = value_of(team_min<L>(least)), y = value_of(team_max<L>(most));
                close = y != none && !(x - y > 4 * error + team_maxf<L>(magnitude) * 0x1p-22f);
            }
            local = 0u;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = (i / VEC * L + lane) * VEC + i % VEC;
                key[i] = e < a.experts ? cells[e] : 0u;
                local = key[i] > local ? key[i] : local;
            }
        }

        // the best, one after another; by sums one more, to see how far it is
        const int rounds = a.slots + (SUMS ? 1 : 0);
        for (int k = 0; k < rounds; ++k) {
            const uint32_t best = team_max<L>(local);
            int at = V;  // the lowest of this lane's that has that key
#pragma unroll
            for (int i = V - 1; i >= 0; --i) at = key[i] == best ? i : at;
            const uint32_t mine = at == V ? ~0u : (uint32_t)((at / VEC * L + lane) * VEC + at % VEC);
            const uint32_t e = team_min<L>(mine);
            const int gone = mine == e ? at : V;
            local = 0u;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                key[i] = i == gone ? 0u : key[i];
                local = key[i] > local ? key[i] : local;
            }
            if (lane == 0) list[k] = {best == 0u ? -1 : (int)e, best};
        }
        wave_sync();
        if constexpr (SUMS) {
            for (int k = lane; k < a.slots; k += L) {
                const float x = value_of(list[k].key), y = value_of(list[k + 1].key);
                close |= y != none && !(x - y > 2 * error + (__builtin_fabsf(x) + __builtin_fabsf(y)) * 0x1p-23f);
            }
            if (team_or<L>(close && live) != 0u) choose_in_64<T, L>(row, a, lane, top, cells64, list);
        }

        // weights: of each chosen logit, by the softmax's or the sigmoid's parts
        float high = none;
        for (int k = lane; k < a.slots; k += L) {
            const int e = list[k].expert;
            const float l = e < 0 ? none : SUMS ? load_logit(row, e) : value_of(list[k].key);
            list[k].key = __builtin_bit_cast(uint32_t, l);  // from here on the logit
            high = __builtin_fmaxf(high, l);
        }
        float total = 1.0f;
        if (a.normalize) {
            high = team_maxf<L>(high);
            if (a.sigmoid) high = __builtin_fminf(high, 0.0f);
            total = 0.0f;
            for (int k = lane; k < a.slots; k += L)
                if (list[k].expert >= 0) {
                    const float l = __builtin_bit_cast(float, list[k].key);
                    total += a.sigmoid ? sigmoid_above(l, high) : expf(l - high);
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
                const float l = __builtin_bit_cast(float, list[k].key);
                const float s = a.sigmoid ? sigmoid_above(l, high) : expf(l - high);
                store_scalar(a.weights, a.weight_type, at, e < 0 ? 0.0f : a.scale * (s / total));
            }
        wave_sync();  // the list is used again
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
// has its share.
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
    const float none = -__builtin_inff();

    for (int64_t t = (int64_t)blockIdx.x * kTeams + team; t - team < a.tokens; t += kMaxGridX * kTeams) {
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
                s[i] = s[i] == none ? 0.0f : expf(s[i] - top);
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

        // each place's expert and logit; then its share
        float high = none;
        for (int k = lane; k < a.slots; k += L) {
            const int64_t at = t * a.slots + k;
            int64_t id = -1;
            if (live) id = a.wide_ids ? ((const int64_t *)a.ids)[at] : ((const int32_t *)a.ids)[at];
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
                dot += w * (a.scale * load_scalar(a.grad_weights, a.weight_type, t * a.slots + k));
            }
        dot = team_sum<L>(dot);
        for (int k = lane; k < a.slots; k += L)
            if (list[k].expert >= 0) {
                const float l = list[k].by, w = (a.sigmoid ? sigmoid_above(l, high) : expf(l - high)) / total;
                const float g = a.scale * load_scalar(a.grad_weights, a.weight_type, t * a.slots + k);
                const float d = w * (a.normalize ? g - dot : g);
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
#pragma unroll
            for (int j = 0; j < V / VEC; ++j) {
                const Col col = col_of<T>(a.experts, (int64_t)(j * L + lane) * VEC);
                float d[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    d[i] = cells[(j * L + lane) * VEC + i];
                    if constexpr (WHOLE) {
                        const float p = s[j * VEC + i] / sum;
                        d[i] -= p == 0.0f ? 0.0f : p * dot;
                    }
                }
                store_col<T>(out, pack<T>(d), col);
            }
        }
        wave_sync();
    }
}

}  // namespace lrs_choose
