// route.hip -- host side of a router's calls of include/lrsort_choose.h: argument checks
// and kernel launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lrsort_choose.h"
#include "route_kernels.hpp"
#include "row_args.hpp"

namespace {

using namespace lrs_choose;

static_assert(kMaxSlots == LRS_MAX_SLOTS && kMaxGroups == LRS_MAX_GROUPS, "limits of the header");

// ------------------------------------------------------------------- routing

// Lanes that serve a token, and logits a lane holds.  16,384 tokens by sigmoid, bias and
// groups of two / bf16 by logits / gradient, in us, and the same with other teams: 64
// experts 10.7 / 4.6 / 5.4 (sixteen lanes 11.6 / 6.1 / 6.2), 128 12.5 / 6.0 / 7.2 (eight of
// 16 logits 14.5 / 5.5 / 7.6), 512 31.3 / 12.5 / 15.3 (64 lanes 32.6 / 16.1 / 17.2); 4,096
// tokens of 1,024 27.7 / 8.3 / 10.7 (32 lanes 29.6 / 7.7 / 11.2); 256: the kernel's comment.
template <int LANES, int LOGITS>
struct Team {
    static constexpr int lanes = LANES, logits = LOGITS;
};

template <typename F>
void with_team(int64_t experts, F &&f)
{
    if (experts <= 64)
        f(Team<8, 8>{});
    else if (experts <= 128)
        f(Team<16, 8>{});
    else if (experts <= 256)
        f(Team<16, 16>{});
    else if (experts <= 512)
        f(Team<32, 16>{});
    else if (experts <= 1024)
        f(Team<64, 16>{});
    else
        f(Team<64, 32>{});
}

template <typename TEAM>
dim3 team_grid(int64_t tokens)
{
    const int64_t teams = kTeamThreads / TEAM::lanes, tiles = (tokens + teams - 1) / teams;
    return dim3((unsigned)std::min(tiles, kMaxGridX), (unsigned)((tiles + kMaxGridX - 1) / kMaxGridX));
}

bool score_ok(lrs_score_type s) { return s == LRS_SCORE_SOFTMAX || s == LRS_SCORE_SIGMOID; }

bool route_sizes_ok(int64_t tokens, int64_t experts, int64_t slots, int64_t ld)
{
    return slots_ok(tokens, slots) && slots <= kMaxSlots && experts >= 0 && experts <= LRS_MAX_EXPERTS &&
           shape_ok(tokens, experts, ld);
}

constexpr int team_align(int64_t bytes) { return (int)((bytes + 15) / 16 * 16); }

}  // namespace

LRS_API lrs_status lrs_route_tokens(lrs_row_type type, const void *d_logits, int64_t ld_logits, int64_t tokens,
                                    int64_t experts, int64_t slots, lrs_score_type score, const float *d_bias,
                                    int64_t num_groups, int64_t kept_groups, lrs_group_score group_score, int normalize,
                                    float scale, lrs_id_type id_type, void *d_ids, lrs_row_type weight_type,
                                    void *d_weights, hipStream_t stream)
{
    if (!type_ok(type) || !type_ok(id_type) || (d_weights && !type_ok(weight_type)) || !score_ok(score) ||
        (group_score != LRS_GROUP_MAX && group_score != LRS_GROUP_TOP2) ||
        !route_sizes_ok(tokens, experts, slots, ld_logits) || num_groups < 1 || num_groups > kMaxGroups ||
        kept_groups < 1 || kept_groups > num_groups || experts % num_groups != 0 ||
        slots > kept_groups * (experts / num_groups))
        return LRS_ERR_INVALID_ARG;
    const int64_t b = bytes_of(type), n = tokens * slots;
    if (n == 0) return LRS_OK;
    const Span logits = matrix_of(d_logits, tokens, experts, ld_logits, b);
    const Span bias = vector_of(d_bias, d_bias ? experts : 0, 4), ids = vector_of(d_ids, n, bytes_of(id_type));
    const Span w = vector_of(d_weights, d_weights ? n : 0, bytes_of(weight_type));
    if (!array_ok(logits, b) || !array_ok(bias, 4) || !array_ok(ids, bytes_of(id_type)) ||
        !array_ok(w, bytes_of(weight_type)) || overlap(ids, logits) || overlap(ids, bias) || overlap(w, logits) ||
        overlap(w, bias) || overlap(w, ids))
        return LRS_ERR_INVALID_ARG;
    const bool grouped = kept_groups < num_groups;
    const bool top2 = grouped && group_score == LRS_GROUP_TOP2, sums = d_bias != nullptr || top2;
    const int size = (int)(experts / num_groups);
    const uint8_t sigmoid = score != LRS_SCORE_SIGMOID ? 0 : d_bias != nullptr ? 1 : 2;
    Route a{d_bias, d_ids, d_weights, scale, (int)tokens, (int16_t)experts, (int16_t)size, (int16_t)num_groups,
            (int16_t)kept_groups, (uint8_t)slots, sigmoid, top2, normalize != 0, id_type == LRS_ID_I64,
            (uint8_t)weight_type, 0, 0};
    // a token's list of the chosen, and its scores and groups where they are needed
    const int cells = sums || b == 4 ? 8 : grouped ? 4 : 0;
    const int team_bytes = team_align((slots + 2) * (int64_t)sizeof(Chosen) + cells * (experts + num_groups));
    return with_type(type, [&](auto elem) {
        using T = decltype(elem);
        with_team(experts, [&](auto team) {
            using TEAM = decltype(team);
            const int lanes = size / kVec<T>;
            if (size % kVec<T> == 0 && (lanes & (lanes - 1)) == 0 && lanes <= std::min(TEAM::lanes, 16))
                a.lane_groups = (uint8_t)lanes, a.lane_groups_log2 = (uint8_t)__builtin_ctz((unsigned)lanes);
            const unsigned lds = (unsigned)team_bytes * (kTeamThreads / TEAM::lanes);
            with_bool(sums, [&](auto by_sums) {
                route_kernel<T, TEAM::lanes, TEAM::logits, by_sums.value>
                    <<<team_grid<TEAM>(tokens), kTeamThreads, lds, stream>>>((const T *)d_logits, ld_logits, a,
                                                                            team_bytes);
            });
        });
        return launched();
    });
}

LRS_API lrs_status lrs_route_tokens_grad(lrs_row_type type, const void *d_logits, int64_t ld_logits, int64_t tokens,
                                         int64_t experts, int64_t slots, lrs_score_type score, int normalize,
                                         float scale, lrs_id_type id_type, const void *d_ids, lrs_row_type weight_type,
                                         const void *d_grad_weights, void *d_grad_logits, int64_t ld_grad_logits,
                                         hipStream_t stream)
{
    if (!type_ok(type) || !type_ok(id_type) || !type_ok(weight_type) || !score_ok(score) ||
        !route_sizes_ok(tokens, experts, slots, ld_logits) || !shape_ok(tokens, experts, ld_grad_logits))
        return LRS_ERR_INVALID_ARG;
    const int64_t b = bytes_of(type), n = tokens * slots;
    if (tokens == 0 || experts == 0) return LRS_OK;
    const Span logits = matrix_of(d_logits, tokens, experts, ld_logits, b);
    const Span grad = matrix_of(d_grad_logits, tokens, experts, ld_grad_logits, b);
    const Span ids = vector_of(d_ids, n, bytes_of(id_type)), gw = vector_of(d_grad_weights, n, bytes_of(weight_type));
    const bool in_place = logits.at == grad.at && logits.step == grad.step;
    if (!array_ok(logits, b) || !array_ok(grad, b) || !array_ok(ids, bytes_of(id_type)) ||
        !array_ok(gw, bytes_of(weight_type)) || (!in_place && overlap(grad, logits)) || overlap(grad, ids) ||
        overlap(grad, gw))
        return LRS_ERR_INVALID_ARG;
    const RouteGrad a{d_ids, d_grad_weights, scale, (int)tokens, (int16_t)experts, (uint8_t)slots,
                      score == LRS_SCORE_SIGMOID, normalize != 0, id_type == LRS_ID_I64, (uint8_t)weight_type};
    return with_type(type, [&](auto elem) {
        using T = decltype(elem);
        with_team(experts, [&](auto team) {
            using TEAM = decltype(team);
            const int team_bytes = team_align(TEAM::lanes * TEAM::logits * 4 + slots * ((int64_t)sizeof(Share) + 4));
            const unsigned lds = (unsigned)team_bytes * (kTeamThreads / TEAM::lanes);
            with_bool(score == LRS_SCORE_SOFTMAX && !normalize, [&](auto whole) {
                route_grad_kernel<T, TEAM::lanes, TEAM::logits, whole.value>
                    <<<team_grid<TEAM>(tokens), kTeamThreads, lds, stream>>>(
                        (const T *)d_logits, ld_logits, (T *)d_grad_logits, ld_grad_logits, a, team_bytes);
            });
        });
        return launched();
    });
}
