// rows.hip -- host side of include/lrsort_rows.h: argument checks, temp-storage
// layout and kernel launches on the caller's stream.  Where keys have to be
// sorted it calls the library's own sort (lrs_sort_digits) with part of the
// caller's temp storage.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "group_kernels.hpp"
#include "lrsort.h"
#include "lrsort_rows.h"
#include "row_args.hpp"
#include "row_kernels.hpp"

namespace {

using namespace lrs_rows;

// ------------------------------------------------------------------ launches

// Lanes per row: as many as its vectors, a power of two up to a workgroup.
struct Tiling {
    int tx_log2;
    int64_t vecs, row_tiles, col_tiles;
};

Tiling tiling_of(int64_t rows, int64_t cols, int vec)
{
    Tiling t;
    t.vecs = (cols + vec - 1) / vec;
    t.tx_log2 = 0;
    while ((1 << t.tx_log2) < kThreads && (1 << t.tx_log2) < t.vecs) ++t.tx_log2;
    const int64_t ty = kThreads >> t.tx_log2;
    t.row_tiles = (rows + ty - 1) / ty;
    t.col_tiles = (t.vecs + (1 << t.tx_log2) - 1) >> t.tx_log2;
    return t;
}

dim3 grid_of(const Tiling &t)
{
    return dim3((unsigned)std::min(t.col_tiles, kMaxGridX), (unsigned)std::min(t.row_tiles, kMaxGridY));
}

bool wave_row(const Tiling &t) { return (1 << t.tx_log2) >= kWave; }

unsigned flat_grid(int64_t n)
{
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>((n + kThreads - 1) / kThreads, 8192));
}

// Times here and below: rows of 4096 bf16, 8 slots a token, calls back to back.
//
// Below this many workgroups (eight a CU) the chip is not full, and a token's slots
// are taken at once: the gradient of 128 tokens in 10.4 us instead of 15.5, of 512 in
// 20.6 instead of 23.3 and their sum in 8.1 instead of 9.5.  Above it slot by slot:
// 16,384 tokens, sum 200 us instead of 217, gradient 442 instead of 465; 4,096 tokens,
// gradient 111 instead of 119 (more rows open at once cost HBM more than they hide).
// At 1,024 tokens the limit is off by some us either way: the gradient takes 35.3 at
// once and 29.8 slot by slot, the sum 16.8 slot by slot and 13.8 at once.
constexpr int64_t kFewTiles = 2048;

// More bytes than the L2s hold (32 MB) go past them: 16,384 tokens, sum 200 us instead
// of 230, gradient 442 instead of 456; 2,048 tokens, 28 instead of 33 and 64 instead of
// 69; 512 tokens (38 MB) the same either way, 1,024 (75 MB) 17 instead of 14 and 35
// instead of 37.  The bytes are those of all slots, also of those without a position:
// a rank with a share of the experts is taken for one that holds them all.
bool streams(int64_t bytes) { return bytes > ((int64_t)32 << 20); }

// A gradient of more bytes than the last-level cache is read past the L2s; a smaller
// one may still be there from the kernel that wrote it.
constexpr int64_t kLastCacheBytes = (int64_t)256 << 20;

// LDS that a dispatch asks for and does not use, so that six workgroups fit a CU
// and not eight: fewer rows are being written at once.  16,384 tokens in 225 us
// instead of 244, 4,096 in 58 instead of 60; rows of 4 KB the same, and small calls
// too.
constexpr unsigned kDispatchLds = 26 * 1024;

// ------------------------------------------------------------------ grouping

// Few ids are ordered by counting passes of this file's own, the others by the
// library's sort.  (Times of orders: a call's on the GPU, calls back to back in a
// captured graph, ids uniform.)
//
// A grouping of up to 2048 groups and 2^20 ids takes one pass: 262,144 ids of 256
// groups 14 us, by the sort 32, 2^20 ids 24 and 47, 2^21 57 and 62; of 2048 groups 25
// and 44, 59 and 63, 179 and 82 (and if all ids are equal, 22 and 27, 50 and 38).
constexpr int kFewBins = 513, kManyBins = 2049;
constexpr int64_t kDirectGroups = kManyBins - 1, kDirectSlots = 1 << 20;

// Blocks of 1024 slots, or of 4096 where those would be many (a block reads every
// block's counts; a wave's ranking is what they share): 131,072 ids of 256 groups in
// 11.8 us by 1024, 12.5 by 4096, 262,144 in 16.5 and 14.1; of 2048 groups 32,768 ids in
// 14.5 and 15.9, 65,536 in 19.1 and 17.2.  Up to 12K slots the blocks count one
// another's slots and need no count launch (which is 3 us of the host's too): 8,192 ids
// of 256 groups in 7.0 us instead of 7.9, 12,288 in 8.1 instead of 8.9, 16,384 in 9.3
// instead of 7.6; of 8 groups 8,192 in 6.3 either way, 12,288 in 7.5 instead of 6.4; of
// 2048 groups 12,288 in 11.0 instead of 13.5, 24,576 in 14.6 instead of 13.4.
constexpr int64_t kSelfCountSlots = 12 * kPlaceThreads;

int place_items(int64_t n, int64_t bins) { return n <= (bins <= kFewBins ? 128 : 32) * kPlaceThreads ? 1 : 4; }
int place_blocks(int64_t n, int items)
{
    const int64_t slots = (int64_t)kPlaceThreads * items;
    return (int)std::max<int64_t>(1, (n + slots - 1) / slots);
}

template <int MAX_BINS, int ITEMS, typename SRC>
lrs_status run_pass(const SRC &src, const Pass &ps, uint32_t *counts, const PlaceOut &out, uint32_t *clear,
                    hipStream_t stream)
{
    const int blocks = place_blocks(ps.n, ITEMS);
    const bool count = blocks > 1 && ps.n > kSelfCountSlots;
    if (count) {
        count_kernel<SRC, MAX_BINS, ITEMS><<<blocks, kPlaceThreads, 0, stream>>>(src, ps, counts, clear);
        const lrs_status st = launched();
        if (st != LRS_OK) return st;
    }
    place_kernel<SRC, MAX_BINS, ITEMS><<<blocks, kPlaceThreads, 0, stream>>>(
        src, ps, count ? counts : nullptr, blocks, out, count ? nullptr : clear);
    return launched();
}

// A pass in blocks of 1024 slots: every pass of an order of ids, which are 131,072 at
// most, and of digits above nine bits 32,768.
template <typename SRC>
lrs_status run_pass(const SRC &src, const Pass &ps, uint32_t *counts, const PlaceOut &out, uint32_t *clear,
                    hipStream_t stream)
{
    return ps.bins <= kFewBins ? run_pass<kFewBins, 1>(src, ps, counts, out, clear, stream)
                               : run_pass<kManyBins, 1>(src, ps, counts, out, clear, stream);
}

int bits_of(int64_t values)  // bits that hold 0..values - 1
{
    int bits = 0;
    while (((int64_t)1 << bits) < values) ++bits;
    return bits;
}

// Temp storage of an order of ids: keys and indices before and after sorting, and the
// sort's own or the passes' counts.
struct GroupLayout {
    size_t off_keys = 0, off_index = 0, off_sorted = 0, off_order = 0, off_sort = 0, sort_bytes = 0, total = 0;
    int bits = 0;
};

// An embedding's ids are ordered by passes of up to eleven bits up to kDirectIds of
// them: 131,072 of 65,536 ids 30 us, by the sort 44, of 1,000,000 ids 41 and 53, all
// equal 26 and 40.  262,144 would take 41 and 49, 50 and 70, 33 and 32; 524,288 80 and
// 58, 75 and 80.  Up to kOrderSlots one block has all passes.
constexpr int64_t kDirectIds = 1 << 17, kOrderSlots = 4 * kPlaceThreads;
int passes_of(int bits, int digit) { return (std::max(bits, 1) + digit - 1) / digit; }

// Bits of a pass's digit.  Digits of eleven bits save a launch or two in some orders,
// and the more slots, the more their counts cost: 12,000 keys of 11 bits added up in
// 31.6 us with one pass, 38.4 with two; of 19 bits 36 with two, 43.5 with three; 32,768
// of 10 bits 28.5 and 31.3, but of 22 bits (digits of eleven) 56 and 50.5; 65,536 keys
// of 10 bits 33.5 and 32.  (Up to kOrderSlots the passes share a launch.)
int digit_bits(int64_t n, int bits)
{
    const int most = n <= kOrderSlots ? 9 : n <= 16 * kPlaceThreads ? 11 : n <= 32 * kPlaceThreads ? 10 : 9;
    return passes_of(bits, passes_of(bits, most));
}

lrs_status group_layout(int64_t n, int64_t groups, GroupLayout *L)
{
    L->bits = bits_of(groups + 1);  // keys are 0..groups
    const size_t words = align_up((size_t)(n + kKeyPad) * 4);  // (the sums read some words past the end)
    size_t off = 0;
    L->off_keys = off, off += words;
    L->off_index = off, off += words;
    L->off_sorted = off, off += words;
    L->off_order = off, off += words;
    L->off_sort = off;
    lrs_status st = LRS_OK;
    if (n <= kDirectIds) {
        L->sort_bytes = ((size_t)place_blocks(n, 1) * 4) << digit_bits(n, L->bits);
    } else {
        // the size depends on n and the bit range alone: any distinct pointers will do
        const uintptr_t some = (uintptr_t)1 << 40;
        st = lrs_sort_digits(LRS_KEY_U32, 8, nullptr, &L->sort_bytes, (const void *)some, (const uint32_t *)(2 * some),
                             (void *)(3 * some), (uint32_t *)(4 * some), n, 0, L->bits, nullptr);
    }
    L->total = off + L->sort_bytes;
    return st;
}

// The sorted keys and their indices (in `order` if that is not NULL, else in temp
// storage).  The first kernel sets *clear to zero, where it is given.
template <typename ID>
lrs_status sort_ids(const GroupLayout &L, char *temp, const void *ids, int64_t n, int64_t first, int64_t groups,
                    int32_t *order, const uint32_t **sorted, const uint32_t **index, uint32_t *clear,
                    hipStream_t stream)
{
    uint32_t *keys = (uint32_t *)(temp + L.off_keys), *at = (uint32_t *)(temp + L.off_index);
    uint32_t *out = (uint32_t *)(temp + L.off_sorted);
    uint32_t *ord = order != nullptr ? (uint32_t *)order : (uint32_t *)(temp + L.off_order);
    *sorted = out, *index = ord;
    if (n == 0) return LRS_OK;
    const IdSource<ID> src{(const ID *)ids, first, (uint32_t)groups};
    if (n <= kDirectIds) {
        const int width = digit_bits(n, L.bits), passes = passes_of(L.bits, width);
        if (n <= kOrderSlots) {
            auto *k = n <= kPlaceThreads ? order_kernel<ID, kFewBins, 1> : order_kernel<ID, kFewBins, 4>;
            k<<<1, kPlaceThreads, 0, stream>>>(src, (int)n, L.bits, width, out, ord, clear);
            return launched();
        }
        uint32_t *counts = (uint32_t *)(temp + L.off_sort);
        for (int p = 0; p < passes; ++p) {
            const int shift = p * width, bits = std::min(width, std::max(L.bits, 1) - shift);
            const Pass ps{(int)n, (1u << bits) - 1u, (uint16_t)(1u << bits), (uint8_t)shift, (uint8_t)bits};
            // the passes alternate between the two pairs of arrays so that the last
            // one writes the sorted ones
            const bool to_out = (passes - 1 - p) % 2 == 0;
            const PlaceOut dst = to_out ? PlaceOut{out, ord, nullptr, nullptr} : PlaceOut{keys, at, nullptr, nullptr};
            const PairSource from = to_out ? PairSource{keys, at} : PairSource{out, ord};
            const lrs_status st = p == 0 ? run_pass(src, ps, counts, dst, clear, stream)
                                         : run_pass(from, ps, counts, dst, nullptr, stream);
            if (st != LRS_OK) return st;
        }
        return LRS_OK;
    }
    group_keys_kernel<ID><<<flat_grid(n), kThreads, 0, stream>>>((const ID *)ids, (int)n, first, (uint32_t)groups, keys,
                                                                at, clear);
    const lrs_status st = launched();
    if (st != LRS_OK) return st;
    size_t bytes = L.sort_bytes;
    return lrs_sort_digits(LRS_KEY_U32, 8, temp + L.off_sort, &bytes, keys, at, out, ord, n, 0, L.bits, stream);
}

lrs_status sort_ids(const GroupLayout &L, char *temp, lrs_id_type id_type, const void *ids, int64_t n, int64_t first,
                    int64_t groups, int32_t *order, const uint32_t **sorted, const uint32_t **index, uint32_t *clear,
                    hipStream_t stream)
{
    return id_type == LRS_ID_I32
               ? sort_ids<int32_t>(L, temp, ids, n, first, groups, order, sorted, index, clear, stream)
               : sort_ids<int64_t>(L, temp, ids, n, first, groups, order, sorted, index, clear, stream);
}

template <typename ID>
lrs_status group_direct(const void *ids, int64_t n, int64_t first, int64_t groups, uint32_t *counts, int32_t *order,
                        int32_t *position, int32_t *offsets, hipStream_t stream)
{
    const IdSource<ID> src{(const ID *)ids, first, (uint32_t)groups};
    const Pass ps{(int)n, ~0u, (uint16_t)(groups + 1), 0, (uint8_t)bits_of(groups + 1)};
    const PlaceOut out{nullptr, (uint32_t *)order, position, offsets};
    if (place_items(n, ps.bins) == 1) return run_pass(src, ps, counts, out, nullptr, stream);
    return ps.bins <= kFewBins ? run_pass<kFewBins, 4>(src, ps, counts, out, nullptr, stream)
                               : run_pass<kManyBins, 4>(src, ps, counts, out, nullptr, stream);
}

lrs_status group_entry(void *d_temp, size_t *temp_bytes, lrs_id_type id_type, const void *d_ids, int64_t n,
                       int64_t first, int64_t groups, int32_t *order, int32_t *position, int32_t *offsets,
                       hipStream_t stream)
{
    if (temp_bytes == nullptr || !type_ok(id_type) || !count_ok(n) || !ids_ok(first, groups) || groups >= kMaxCount)
        return LRS_ERR_INVALID_ARG;
    const Span ids = vector_of(d_ids, n, bytes_of(id_type));
    const Span outs[3] = {vector_of(order, order ? n : 0, 4), vector_of(position, position ? n : 0, 4),
                          vector_of(offsets, offsets ? groups + 1 : 0, 4)};
    if (!array_ok(ids, bytes_of(id_type))) return LRS_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i) {
        if (!array_ok(outs[i], 4) || overlap(outs[i], ids)) return LRS_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return LRS_ERR_INVALID_ARG;
    }
    const bool direct = groups <= kDirectGroups && n <= kDirectSlots;
    GroupLayout L;
    lrs_status st = LRS_OK;
    if (direct)
        L.total = n <= kSelfCountSlots
                      ? 0
                      : (size_t)place_blocks(n, place_items(n, groups + 1)) * (size_t)(groups + 1) * 4;
    else
        st = group_layout(n, groups, &L);
    if (st != LRS_OK) return st;
    char *temp;
    st = take_temp(d_temp, temp_bytes, L.total, &temp);
    if (st != LRS_OK || temp == nullptr) return st;
    if (order == nullptr && position == nullptr && offsets == nullptr) return LRS_OK;
    if (direct) {
        if (id_type == LRS_ID_I32)
            return group_direct<int32_t>(d_ids, n, first, groups, (uint32_t *)temp, order, position, offsets, stream);
        return group_direct<int64_t>(d_ids, n, first, groups, (uint32_t *)temp, order, position, offsets, stream);
    }
    const uint32_t *sorted, *index;
    st = sort_ids(L, temp, id_type, d_ids, n, first, groups, order, &sorted, &index, nullptr, stream);
    if (st != LRS_OK || (position == nullptr && offsets == nullptr)) return st;
    group_finish_kernel<<<flat_grid(std::max(n, groups + 1)), kThreads, 0, stream>>>(sorted, index, n, (uint32_t)groups,
                                                                                     position, offsets);
    return launched();
}

}  // namespace

// ------------------------------------------------------------------- exports

LRS_API lrs_status lrs_group_tokens(void *d_temp, size_t *temp_bytes, lrs_id_type id_type, const void *d_ids, int64_t n,
                                    int64_t first_id, int64_t num_groups, int32_t *d_order, int32_t *d_position,
                                    int32_t *d_offsets, hipStream_t stream)
{
    return guarded([&] {
        return group_entry(d_temp, temp_bytes, id_type, d_ids, n, first_id, num_groups, d_order, d_position, d_offsets,
                           stream);
    });
}

LRS_API lrs_status lrs_dispatch_rows(lrs_row_type type, const void *d_x, int64_t ld_x, const int32_t *d_position,
                                     int64_t tokens, int64_t slots, int64_t cols, void *d_rows, int64_t ld_rows,
                                     int64_t num_rows, hipStream_t stream)
{
    if (!type_ok(type) || !slots_ok(tokens, slots) || !shape_ok(tokens, cols, ld_x) ||
        !shape_ok(num_rows, cols, ld_rows))
        return LRS_ERR_INVALID_ARG;
    const int64_t b = bytes_of(type);
    if (tokens == 0 || slots == 0 || cols == 0 || num_rows == 0) return LRS_OK;
    const Span x = matrix_of(d_x, tokens, cols, ld_x, b), rows = matrix_of(d_rows, num_rows, cols, ld_rows, b);
    const Span pos = vector_of(d_position, tokens * slots, 4);
    if (!array_ok(x, b) || !array_ok(rows, b) || !array_ok(pos, 4) || overlap(rows, x) || overlap(rows, pos))
        return LRS_ERR_INVALID_ARG;
    auto run = [&](auto word) {
        using W = decltype(word);
        const Tiling t = tiling_of(tokens, cols, kVec<W>);
        auto *k = wave_row(t) ? dispatch_kernel<W, true> : dispatch_kernel<W, false>;
        k<<<grid_of(t), kThreads, kDispatchLds, stream>>>((const W *)d_x, ld_x, d_position, (int)tokens, (int)slots,
                                                          (int)cols, (uint32_t)num_rows, (W *)d_rows, ld_rows,
                                                          t.tx_log2);
        return launched();
    };
    return b == 4 ? run(uint32_t{}) : run(uint16_t{});
}

LRS_API lrs_status lrs_combine_rows(lrs_row_type type, const void *d_rows, int64_t ld_rows, int64_t num_rows,
                                    const int32_t *d_position, lrs_row_type weight_type, const void *d_weights,
                                    int64_t tokens, int64_t slots, int64_t cols, void *d_y, int64_t ld_y,
                                    hipStream_t stream)
{
    if (!type_ok(type) || (d_weights && !type_ok(weight_type)) || !slots_ok(tokens, slots) ||
        !shape_ok(num_rows, cols, ld_rows) || !shape_ok(tokens, cols, ld_y))
        return LRS_ERR_INVALID_ARG;
    const int64_t b = bytes_of(type), n = tokens * slots;
    if (tokens == 0 || cols == 0) return LRS_OK;
    const Span rows = matrix_of(d_rows, num_rows, cols, ld_rows, b), y = matrix_of(d_y, tokens, cols, ld_y, b);
    const Span pos = vector_of(d_position, n, 4);
    const Span w = vector_of(d_weights, d_weights ? n : 0, bytes_of(weight_type));
    if (!array_ok(rows, b) || !array_ok(y, b) || !array_ok(pos, 4) || !array_ok(w, bytes_of(weight_type)) ||
        overlap(y, rows) || overlap(y, pos) || overlap(y, w))
        return LRS_ERR_INVALID_ARG;
    return with_type(type, [&](auto elem) {
        using T = decltype(elem);
        const Tiling t = tiling_of(tokens, cols, kVec<T>);
        auto pick = [&](auto wave, auto slots_at_once, auto nt) {
            combine_kernel<T, wave.value, slots_at_once.value, nt.value><<<grid_of(t), kThreads, 0, stream>>>(
                (const T *)d_rows, ld_rows, (uint32_t)num_rows, (int)weight_type, d_position, d_weights, (int)tokens,
                (int)slots, (int)cols, t.tx_log2, (T *)d_y, ld_y);
        };
        const bool few = t.row_tiles * t.col_tiles < kFewTiles;
        with_bool(wave_row(t), [&](auto wave) {
            with_bool(streams((n + tokens) * cols * b), [&](auto nt) {
                if (few)
                    pick(wave, std::integral_constant<int, 8>{}, nt);
                else
                    pick(wave, std::integral_constant<int, 1>{}, nt);
            });
        });
        return launched();
    });
}

LRS_API lrs_status lrs_combine_rows_grad(lrs_row_type type, const void *d_grad_y, int64_t ld_grad_y, const void *d_rows,
                                         int64_t ld_rows, int64_t num_rows, const int32_t *d_position,
                                         lrs_row_type weight_type, const void *d_weights, int64_t tokens, int64_t slots,
                                         int64_t cols, void *d_grad_rows, int64_t ld_grad_rows, void *d_grad_weights,
                                         hipStream_t stream)
{
    if (!type_ok(type) || ((d_weights || d_grad_weights) && !type_ok(weight_type)) || !slots_ok(tokens, slots) ||
        !shape_ok(tokens, cols, ld_grad_y) || !shape_ok(num_rows, cols, ld_grad_rows) ||
        (d_grad_weights && !shape_ok(num_rows, cols, ld_rows)))
        return LRS_ERR_INVALID_ARG;
    const int64_t b = bytes_of(type), wb = bytes_of(weight_type), n = tokens * slots;
    if (n == 0) return LRS_OK;
    const Span gy = matrix_of(d_grad_y, tokens, cols, ld_grad_y, b);
    const Span rows = matrix_of(d_rows, d_grad_weights ? num_rows : 0, cols, ld_rows, b);
    const Span gr = matrix_of(d_grad_rows, num_rows, cols, ld_grad_rows, b);
    const Span pos = vector_of(d_position, n, 4), w = vector_of(d_weights, d_weights ? n : 0, wb);
    const Span gw = vector_of(d_grad_weights, d_grad_weights ? n : 0, wb);
    if (!array_ok(gy, b) || !array_ok(rows, b) || !array_ok(gr, b) || !array_ok(pos, 4) || !array_ok(w, wb) ||
        !array_ok(gw, wb))
        return LRS_ERR_INVALID_ARG;
    const bool in_place = !rows.empty() && rows.at == gr.at && rows.step == gr.step;
    if (overlap(gr, gy) || (!in_place && overlap(gr, rows)) || overlap(gr, pos) || overlap(gr, w) || overlap(gw, gy) ||
        overlap(gw, rows) || overlap(gw, gr) || overlap(gw, pos) || overlap(gw, w))
        return LRS_ERR_INVALID_ARG;
    return with_type(type, [&](auto elem) {
        using T = decltype(elem);
        Tiling t = tiling_of(tokens, cols, kVec<T>);
        // Few tokens: a workgroup per slot, so that more of the chip works (grad_y
        // is then read once per slot, from cache).
        const bool few = t.row_tiles < kFewTiles;
        const int64_t at_once = few ? slots : 1;
        const dim3 grid((unsigned)std::min(at_once, kMaxGridX), (unsigned)std::min(t.row_tiles, kMaxGridY));
        with_bool(wave_row(t), [&](auto wave) {
            with_bool(streams((2 * n + tokens) * cols * b), [&](auto nt) {
                combine_grad_kernel<T, wave.value, nt.value><<<grid, kThreads, 0, stream>>>(
                    (const T *)d_grad_y, ld_grad_y, (const T *)d_rows, ld_rows, d_position, d_weights,
                    (T *)d_grad_rows, ld_grad_rows, d_grad_weights, (uint32_t)num_rows, (int)tokens, (int)slots,
                    (int)cols, (int8_t)weight_type, (int8_t)t.tx_log2, few);
            });
        });
        return launched();
    });
}

LRS_API lrs_status lrs_embedding(lrs_row_type type, const void *d_table, int64_t ld_table, int64_t num_ids,
                                 lrs_id_type id_type, const void *d_ids, int64_t n, int64_t first_id, float scale,
                                 int64_t cols, void *d_y, int64_t ld_y, hipStream_t stream)
{
    if (!type_ok(type) || !type_ok(id_type) || !ids_ok(first_id, num_ids) || !shape_ok(num_ids, cols, ld_table) ||
        !shape_ok(n, cols, ld_y))
        return LRS_ERR_INVALID_ARG;
    const int64_t b = bytes_of(type), ib = bytes_of(id_type);
    if (n == 0 || cols == 0) return LRS_OK;
    const Span table = matrix_of(d_table, num_ids, cols, ld_table, b), y = matrix_of(d_y, n, cols, ld_y, b);
    const Span ids = vector_of(d_ids, n, ib);
    if (!array_ok(table, b) || !array_ok(y, b) || !array_ok(ids, ib) || overlap(y, table) || overlap(y, ids))
        return LRS_ERR_INVALID_ARG;
    return with_type(type, [&](auto elem) {
        using T = decltype(elem);
        auto run = [&](auto id) {
            using ID = decltype(id);
            const Tiling t = tiling_of(n, cols, kVec<T>);
            with_bool(wave_row(t), [&](auto wave) {
                with_bool(streams(2 * n * cols * b), [&](auto nt) {
                    embedding_kernel<T, ID, wave.value, nt.value><<<grid_of(t), kThreads, 0, stream>>>(
                        (const T *)d_table, ld_table, (const ID *)d_ids, first_id, (uint32_t)num_ids, (int)n,
                        (int)cols, scale, (T *)d_y, ld_y, t.tx_log2);
                });
            });
            return launched();
        };
        return id_type == LRS_ID_I32 ? run(int32_t{}) : run(int64_t{});
    });
}

namespace {

// How an embedding's gradient cuts the sorted ids: pieces of 16 to 512 slots, so
// many that the chip has some 16384 waves of 64 vectors (more than it holds, so that
// they even out: 65,536 x 4096 added in 220 us, 225 with half as many, 223 with
// twice), and shorter ones where even so a SIMD has no wave (777 x 515 in 17 us
// instead of 25; of 16,384 x 2048 with one id they would make 89 us of 49; rows of 64
// elements gain nothing from pieces shorter still, 11,405 of 717 ids 38 us with 2
// slots and 34 with 8).  And the place of the long runs' partial sums and list.
struct SumLayout {
    int piece = 16;
    int64_t count = 0, cols_padded = 0;
    size_t partial_bytes = 0, list_bytes = 0;
    bool joins() const { return count > 2; }  // a run can go on beyond a piece's next
};

SumLayout sum_layout(int64_t n, int64_t cols, int vec)
{
    SumLayout S;
    const int64_t waves = std::max<int64_t>(1, ((cols + vec - 1) / vec + kWave - 1) / kWave);
    while (S.piece < 512 && n / S.piece > 16384 / waves) S.piece *= 2;
    while (S.piece > 2 && n / S.piece < 1024 / waves) S.piece /= 2;
    S.count = (n + S.piece - 1) / S.piece;
    S.cols_padded = (cols + vec - 1) / vec * vec;
    if (S.joins()) {
        S.partial_bytes = align_up((size_t)S.count * 2 * (size_t)S.cols_padded * 4);
        S.list_bytes = (size_t)(S.count + 1) * 4;
    }
    return S;
}

lrs_status embedding_grad_entry(void *d_temp, size_t *temp_bytes, lrs_row_type type, const void *d_grad_y,
                                int64_t ld_grad_y, lrs_id_type id_type, const void *d_ids, int64_t n, int64_t first,
                                float scale, lrs_row_type grad_type, void *d_grad, int64_t ld_grad, int64_t num_ids,
                                int64_t cols, int accumulate, hipStream_t stream)
{
    if (temp_bytes == nullptr || !type_ok(type) || !type_ok(id_type) || !type_ok(grad_type) ||
        (grad_type != type && grad_type != LRS_ROW_F32) || !ids_ok(first, num_ids) || num_ids >= kMaxCount ||
        !shape_ok(n, cols, ld_grad_y) || !shape_ok(num_ids, cols, ld_grad))
        return LRS_ERR_INVALID_ARG;
    const int64_t b = bytes_of(type), gb = bytes_of(grad_type), ib = bytes_of(id_type);
    const Span gy = matrix_of(d_grad_y, n, cols, ld_grad_y, b), grad = matrix_of(d_grad, num_ids, cols, ld_grad, gb);
    const Span ids = vector_of(d_ids, cols > 0 ? n : 0, ib);
    if (!array_ok(gy, b) || !array_ok(grad, gb) || !array_ok(ids, ib) || overlap(grad, gy) || overlap(grad, ids))
        return LRS_ERR_INVALID_ARG;
    GroupLayout L;
    lrs_status st = group_layout(n, num_ids, &L);
    if (st != LRS_OK) return st;
    const SumLayout S = sum_layout(n, cols, (int)(16 / b));
    char *temp;
    st = take_temp(d_temp, temp_bytes, align_up(L.total) + S.partial_bytes + S.list_bytes, &temp);
    if (st != LRS_OK || temp == nullptr) return st;
    if (num_ids == 0 || cols == 0 || (n == 0 && accumulate)) return LRS_OK;
    const uint32_t *sorted, *index;
    float *partial = (float *)(temp + align_up(L.total));
    uint32_t *list = (uint32_t *)(temp + align_up(L.total) + S.partial_bytes);
    st = sort_ids(L, temp, id_type, d_ids, n, first, num_ids, nullptr, &sorted, &index, S.joins() ? list : nullptr,
                  stream);
    if (st != LRS_OK) return st;
    const Pieces pc{sorted, index, partial, list, (int)n, S.piece, (uint32_t)num_ids, (int)cols};
    return with_type(type, [&](auto elem) {
        using T = decltype(elem);
        auto run = [&](auto gelem) {
            using G = decltype(gelem);
            const GradOut<G> out{(G *)d_grad, ld_grad, scale, accumulate ? 1 : 0};
            const Tiling t = tiling_of(S.count, cols, kVec<T>);
            Tiling fill = tiling_of(num_ids, cols, kVec<G>);
            fill.tx_log2 = std::min(fill.tx_log2, 6);  // a wave per row
            const unsigned sums = (unsigned)std::min(t.row_tiles * t.col_tiles, kMaxGridX);
            const unsigned fills =
                accumulate ? 0u : (unsigned)std::min((num_ids + kFillRows - 1) / kFillRows, kMaxGridX);
            with_bool(wave_row(t), [&](auto wave) {
                with_bool(n * cols * b > kLastCacheBytes, [&](auto nt) {
                    embedding_grad_kernel<T, G, wave.value, nt.value><<<sums + fills, kThreads, 0, stream>>>(
                        (const T *)d_grad_y, ld_grad_y, pc, out, sums, (int16_t)t.tx_log2, (int16_t)fill.tx_log2);
                });
            });
            const lrs_status st = launched();
            if (st != LRS_OK || !S.joins()) return st;
            const int64_t join_tiles = (cols + 4 * kJoinLanes - 1) / (4 * kJoinLanes);
            const unsigned joins = (unsigned)std::min((S.count + 1) / 2 * join_tiles, kMaxJoins);
            embedding_join_kernel<G><<<joins, kThreads, 0, stream>>>(pc, out, (int)S.cols_padded);
            return launched();
        };
        return grad_type == LRS_ROW_F32 ? run(float{}) : run(elem);
    });
}

}  // namespace

LRS_API lrs_status lrs_embedding_grad(void *d_temp, size_t *temp_bytes, lrs_row_type type, const void *d_grad_y,
                                      int64_t ld_grad_y, lrs_id_type id_type, const void *d_ids, int64_t n,
                                      int64_t first_id, float scale, lrs_row_type grad_type, void *d_grad,
                                      int64_t ld_grad, int64_t num_ids, int64_t cols, int accumulate,
                                      hipStream_t stream)
{
    return guarded([&] {
        return embedding_grad_entry(d_temp, temp_bytes, type, d_grad_y, ld_grad_y, id_type, d_ids, n, first_id, scale,
                                    grad_type, d_grad, ld_grad, num_ids, cols, accumulate, stream);
    });
}
