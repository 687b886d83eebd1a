// beam.hip -- host side of beam search's calls of include/lrsort_choose.h: argument
// checks, temp-storage layout and kernel launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "beam_kernels.hpp"
#include "lrsort_choose.h"
#include "row_args.hpp"

namespace {

using namespace lrs_choose;

static_assert(kMaxContinuations == LRS_MAX_BEAM_COUNT && kMaxBeams == LRS_MAX_BEAMS, "limits of the header");

// How the rows of a selection are cut: parts of a workgroup's lanes with `vectors` of 16
// bytes each.
struct ScanLayout {
    int vectors = 8;
    int64_t parts = 0;
    size_t best_bytes = 0, part_bytes = 0;
};

// Fewer vectors a lane until there are so many parts, two workgroups a CU: 64 rows of
// 131,072 bf16 logits in 13.3 us with the join (13.4 for 128 parts, 13.3 for 1024, 13.6
// for 2048), 16 rows in 10.8 (11.3, 11.2, 11.3), of float32 in 11.6 (11.3, 11.8, 15.6), 4
// rows of 32,000 float16 in 9.0 (8.9, 9.0, 9.2), 256 rows of 5,000 in 10.5 (11.8, 10.4,
// 10.3): few parts cost latency, many the join.
constexpr int64_t kScanParts = 512;

ScanLayout scan_layout(int64_t rows, int64_t vocab, int64_t count, int64_t vec)
{
    ScanLayout s;
    auto parts = [&] { return (vocab + kScanThreads * vec * s.vectors - 1) / (kScanThreads * vec * s.vectors); };
    while (s.vectors > 1 && rows * parts() < kScanParts) s.vectors /= 2;
    s.parts = parts();
    s.best_bytes = align_up((size_t)(rows * s.parts * count) * 8);
    s.part_bytes = align_up((size_t)(rows * s.parts) * sizeof(Part));
    return s;
}

lrs_status beam_entry(void *d_temp, size_t *temp_bytes, lrs_row_type type, const void *d_logits, int64_t ld,
                      const float *d_scores, const uint8_t *d_finished, int64_t end_id, int64_t batch, int64_t beams,
                      int64_t vocab, int64_t count, int normalize, float *d_out_scores, int32_t *d_parents,
                      lrs_id_type id_type, void *d_tokens, hipStream_t stream)
{
    if (temp_bytes == nullptr || !type_ok(type) || !type_ok(id_type) || !slots_ok(batch, beams) || vocab < 1 ||
        !slots_ok(beams, vocab) || count < 0 || count > kMaxContinuations || beams > kMaxBeams ||
        !shape_ok(batch * beams, vocab, ld) ||
        (d_finished != nullptr && (end_id < 0 || end_id >= vocab)))
        return LRS_ERR_INVALID_ARG;
    const int64_t b = bytes_of(type), rows = batch * beams, n = batch * count;
    const Span in[3] = {matrix_of(d_logits, rows, vocab, ld, b), vector_of(d_scores, rows, 4),
                        vector_of(d_finished, d_finished ? rows : 0, 1)};
    const Span out[3] = {vector_of(d_out_scores, n, 4), vector_of(d_parents, n, 4),
                         vector_of(d_tokens, n, bytes_of(id_type))};
    if (!array_ok(in[0], b) || !array_ok(in[1], 4) || !array_ok(out[0], 4) || !array_ok(out[1], 4) ||
        !array_ok(out[2], bytes_of(id_type)))
        return LRS_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 3; ++j)
            if (overlap(out[i], in[j])) return LRS_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return LRS_ERR_INVALID_ARG;
    }
    const ScanLayout s = scan_layout(rows, vocab, count, 16 / b);
    char *temp;
    const lrs_status st = take_temp(d_temp, temp_bytes, s.best_bytes + s.part_bytes, &temp);
    if (st != LRS_OK || temp == nullptr || n == 0) return st;
    if (rows > 0) {
        const Scan scan{d_scores, d_finished, (uint64_t *)temp, (Part *)(temp + s.best_bytes), (int)rows, (int)vocab,
                        (int)s.parts, (int)count};
        const int64_t jobs = rows * s.parts;
        const dim3 grid((unsigned)std::min(jobs, kMaxGridX), (unsigned)((jobs + kMaxGridX - 1) / kMaxGridX));
        const lrs_status done = with_type(type, [&](auto elem) {
            using T = decltype(elem);
            with_bool(normalize != 0, [&](auto sum) {
                auto run = [&](auto vectors) {
                    beam_scan_kernel<T, sum.value, vectors.value>
                        <<<grid, kScanThreads, 0, stream>>>((const T *)d_logits, ld, scan);
                };
                if (s.vectors == 8)
                    run(std::integral_constant<int, 8>{});
                else if (s.vectors == 4)
                    run(std::integral_constant<int, 4>{});
                else if (s.vectors == 2)
                    run(std::integral_constant<int, 2>{});
                else
                    run(std::integral_constant<int, 1>{});
            });
            return launched();
        });
        if (done != LRS_OK) return done;
    }
    uint8_t token_bits = 0;
    while (vocab > (int64_t)1 << token_bits) ++token_bits;
    const Join join{d_scores, d_finished, (const uint64_t *)temp, (const Part *)(temp + s.best_bytes), d_out_scores,
                    d_parents, d_tokens, (int)beams, (int)s.parts, (int)count, (int)end_id,
                    normalize != 0, id_type == LRS_ID_I64, token_bits};
    const dim3 searches((unsigned)std::min(batch, kMaxGridX), (unsigned)((batch + kMaxGridX - 1) / kMaxGridX));
    beam_join_kernel<<<searches, kJoinThreads, 0, stream>>>(join, (int)batch);
    return launched();
}

// States of more bytes than the last-level cache keeps beside what is written are read past
// the caches: of 16 searches of 8 beams (537 MB) in place in 133 us instead of 149, into
// others in 153 instead of 159, 201 MB in place in 52 instead of 57.  134 MB would take 35
// instead of 32, and 67 MB written eight times over 108 instead of 87.  (Not narrow rows of
// more than 16 beams in place, where a lane loads a state for each of its 64 beams, a
// needed one again for those that need none: from the caches.)
constexpr int64_t kReadPastBytes = (int64_t)160 << 20;

// A state's memory from its first to its last byte, and whether its rows lie apart.
struct Extent {
    bool ok, apart;
    int64_t bytes;
};

Extent extent_of(const lrs_beam_layout &l, int64_t outer, int64_t batch, int64_t beams, int64_t middle, int64_t rows,
                 int64_t row_bytes)
{
    struct Dim {
        int64_t step, count;
    } d[5] = {{l.outer_step, outer}, {l.batch_step, batch}, {l.beam_step, beams}, {l.middle_step, middle},
              {l.row_step, rows}};
    std::sort(d, d + 5, [](const Dim &a, const Dim &b) { return a.step < b.step; });
    Extent e{true, true, 0};
    __int128 end = row_bytes;
    for (const Dim &x : d) {
        if (x.count <= 1) continue;
        if (x.step < 0) e.ok = false;
        if (x.step < end) e.apart = false;
        end += (__int128)(x.count - 1) * x.step;
    }
    if (end > ((__int128)1 << 56)) e.ok = false;
    e.bytes = e.ok ? (int64_t)end : 0;
    return e;
}

bool same_steps(const lrs_beam_layout &a, const lrs_beam_layout &b, int64_t outer, int64_t batch, int64_t beams,
                int64_t middle, int64_t rows)
{
    return (outer <= 1 || a.outer_step == b.outer_step) && (batch <= 1 || a.batch_step == b.batch_step) &&
           (beams <= 1 || a.beam_step == b.beam_step) && (middle <= 1 || a.middle_step == b.middle_step) &&
           (rows <= 1 || a.row_step == b.row_step);
}

}  // namespace

LRS_API lrs_status lrs_beam_select(void *d_temp, size_t *temp_bytes, lrs_row_type type, const void *d_logits,
                                   int64_t ld_logits, const float *d_scores, const uint8_t *d_finished, int64_t end_id,
                                   int64_t batch, int64_t beams, int64_t vocab, int64_t count, int normalize,
                                   float *d_out_scores, int32_t *d_parents, lrs_id_type id_type, void *d_tokens,
                                   hipStream_t stream)
{
    return beam_entry(d_temp, temp_bytes, type, d_logits, ld_logits, d_scores, d_finished, end_id, batch, beams, vocab,
                      count, normalize, d_out_scores, d_parents, id_type, d_tokens, stream);
}

LRS_API lrs_status lrs_beam_reorder(const void *d_in, const lrs_beam_layout *in_layout, void *d_out,
                                    const lrs_beam_layout *out_layout, const int32_t *d_parents, int64_t outer,
                                    int64_t batch, int64_t beams, int64_t count, int64_t middle, int64_t rows,
                                    int64_t row_bytes, hipStream_t stream)
{
    if (in_layout == nullptr || out_layout == nullptr || !count_ok(outer) || !slots_ok(batch, beams) ||
        !slots_ok(batch, count) || !count_ok(middle) || !count_ok(rows) || row_bytes < 0 ||
        row_bytes > ((int64_t)1 << 56) ||
        (__int128)outer * batch * middle * rows > kMaxCount)
        return LRS_ERR_INVALID_ARG;
    if (outer == 0 || batch == 0 || count == 0 || middle == 0 || rows == 0 || row_bytes == 0) return LRS_OK;
    const Extent in = extent_of(*in_layout, outer, batch, beams, middle, rows, row_bytes);
    const Extent out = extent_of(*out_layout, outer, batch, count, middle, rows, row_bytes);
    if (!in.ok || !out.ok || !out.apart) return LRS_ERR_INVALID_ARG;
    const Span from = vector_of(d_in, beams > 0 ? in.bytes : 0, 1), to = vector_of(d_out, out.bytes, 1);
    const Span parents = vector_of(d_parents, batch * count, 4);
    const bool in_place = from.at == to.at && same_steps(*in_layout, *out_layout, outer, batch, std::max(beams, count),
                                                          middle, rows);
    if (!array_ok(from, 1) || !array_ok(to, 1) || !array_ok(parents, 4) || overlap(to, parents) ||
        // (in place more beams before than after may share memory where those after do not)
        (in_place ? count > kMaxContinuations || !in.apart : overlap(to, from)))
        return LRS_ERR_INVALID_ARG;

    const int word = row_bytes % 4 == 0 ? 4 : row_bytes % 2 == 0 ? 2 : 1;
    Reorder a{};
    a.vecs = row_bytes / 16;
    a.words = (int8_t)(row_bytes % 16 / word);
    a.all_rows = (int)(outer * batch * middle * rows);
    a.rows = (int)rows, a.middle = (int)middle, a.batch = (int)batch, a.beams = (int)beams, a.count = (int)count;
    const int64_t lanes = std::max<int64_t>(a.vecs, a.words);
    while ((1 << a.tx_log2) < kThreads && (1 << a.tx_log2) < lanes) ++a.tx_log2;
    a.in_place = in_place;
    // (a kernel for many beams in narrow rows loads some state for every place and drops what
    // no parent names: without beams before the step there is none, and it loads from the new
    // ones)
    const lrs_beam_layout &il = beams > 0 ? *in_layout : *out_layout, &ol = *out_layout;
    const char *in_at = (const char *)(beams > 0 ? d_in : d_out);
    const Places src{il.outer_step, il.batch_step, il.beam_step, il.middle_step, il.row_step};
    const Places dst{ol.outer_step, ol.batch_step, ol.beam_step, ol.middle_step, ol.row_step};
    a.tiles = (a.vecs + (1 << a.tx_log2) - 1) >> a.tx_log2;
    const int64_t col_tiles = a.tiles + (a.words > 0);
    const int64_t row_tiles = ((int64_t)a.all_rows + (kThreads >> a.tx_log2) - 1) / (kThreads >> a.tx_log2);
    const dim3 grid((unsigned)std::min(col_tiles, kMaxGridX), (unsigned)std::min(row_tiles, kMaxGridY),
                    (unsigned)((row_tiles + kMaxGridY - 1) / kMaxGridY));
    const __int128 read_bytes = (__int128)a.all_rows * row_bytes * std::min(beams, count);
    auto run = [&](auto w, auto most, auto wave) {
        auto launch = [&](auto nt) {
            reorder_kernel<decltype(w), most.value, wave.value, nt.value>
                <<<grid, kThreads, 0, stream>>>(in_at, (char *)d_out, d_parents, src, dst, a);
        };
        if constexpr (most.value > 16 && !wave.value)
            launch(std::false_type{});
        else
            with_bool(read_bytes >= kReadPastBytes, launch);
    };
    auto with_word = [&](auto most, auto wave) {
        if (word == 4)
            run(Word4{}, most, wave);
        else if (word == 2)
            run(Word2{}, most, wave);
        else
            run(Word1{}, most, wave);
    };
    // MOST, by the beams.  A wave's row: 22 MB of 4 beams in 4.9 us with 4 and 5.4 with 16,
    // 537 MB of 8 beams in 133 with 16, which takes 94 registers; with 64 it is 255, and 537
    // MB of 32 take 157.  Narrower rows: 67 MB of 8 beams in 17.9 with 8 and 22.7 with 16.
    // Beams behind MOST follow one after another, but in place all are held at once.
    if ((1 << a.tx_log2) >= kWave) {
        constexpr std::true_type wave{};
        if (count <= 4)
            with_word(std::integral_constant<int, 4>{}, wave);
        else if (count <= 16 || !in_place)
            with_word(std::integral_constant<int, 16>{}, wave);
        else
            with_word(std::integral_constant<int, 64>{}, wave);
    } else {
        constexpr std::false_type wave{};
        if (count <= 8)
            with_word(std::integral_constant<int, 8>{}, wave);
        else if (count <= 16 || !in_place)
            with_word(std::integral_constant<int, 16>{}, wave);
        else
            with_word(std::integral_constant<int, 64>{}, wave);
    }
    return launched();
}
