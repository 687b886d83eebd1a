// row_args.hpp -- what the host sides of the row operators and of the operators that
// choose share: checks of arguments (arrays, matrices, overlap), the two-phase temp
// storage convention, types and truth values as constants.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "lrsort.h"
#include "lrsort_rows.h"
#include "row_vectors.hpp"

#define LRS_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace lrs_rows;

constexpr size_t kAlign = 256;
constexpr int64_t kMaxCount = 0x7FFFFFFFll;  // positions and offsets are int32

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// ------------------------------------------------------------------- checks

inline bool type_ok(lrs_row_type t) { return t == LRS_ROW_F32 || t == LRS_ROW_BF16 || t == LRS_ROW_F16; }
inline bool type_ok(lrs_id_type t) { return t == LRS_ID_I32 || t == LRS_ID_I64; }
inline int64_t bytes_of(lrs_row_type t) { return t == LRS_ROW_F32 ? 4 : 2; }
inline int64_t bytes_of(lrs_id_type t) { return t == LRS_ID_I32 ? 4 : 8; }
inline bool count_ok(int64_t n) { return n >= 0 && n <= kMaxCount; }

// Ids [first, first + count) have to exist as int64.
inline bool ids_ok(int64_t first, int64_t count) { return count_ok(count) && first <= INT64_MAX - count; }

// A matrix argument: `rows` rows of `row` bytes, `step` bytes apart.  A vector is a
// matrix of one row.
struct Span {
    uintptr_t at;
    int64_t rows, row, step;
    bool empty() const { return rows == 0 || row == 0; }
    __int128 extent() const { return (__int128)(rows - 1) * step + row; }
};

inline Span vector_of(const void *p, int64_t n, int64_t bytes) { return {(uintptr_t)p, 1, n * bytes, n * bytes}; }
inline Span matrix_of(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t bytes)
{
    // (one row has no stride, and ld is checked before it is multiplied)
    return {(uintptr_t)p, rows, cols * bytes, rows > 1 ? ld * bytes : cols * bytes};
}

// Strides and sizes that leave address arithmetic well inside 63 bits.
inline bool shape_ok(int64_t rows, int64_t cols, int64_t ld)
{
    if (!count_ok(rows) || !count_ok(cols)) return false;
    if (rows <= 1 || cols == 0) return true;
    return ld >= cols && (__int128)rows * ld <= ((__int128)1 << 56);
}

// The array is there and aligned, or empty.
inline bool array_ok(const Span &s, int64_t bytes) { return s.empty() || (s.at != 0 && s.at % bytes == 0); }

// Whether two arrays share memory: exact where their rows are equally far apart or one
// has a single row (columns of one buffer share none); matrices of other strides do if
// their extents meet.  Row i of a and row j of b meet if the distance between them, d +
// (j - i) * step, is above -b.row and below a.row: the first j - i above decides.
inline bool overlap(const Span &a, const Span &b)
{
    if (a.empty() || b.empty() || a.at == 0 || b.at == 0) return false;
    const __int128 d = (__int128)b.at - (__int128)a.at;
    if (d >= a.extent() || -d >= b.extent()) return false;
    if (a.rows > 1 && b.rows > 1 && a.step != b.step) return true;
    const __int128 step = a.rows > 1 ? a.step : b.step;
    const __int128 above = -b.row - d;  // (j - i) * step has to be more
    __int128 by = above >= 0 ? above / step + 1 : -((-above - 1) / step);
    by = std::max<__int128>(by, 1 - a.rows);
    return by < b.rows && d + by * step < a.row;
}

inline lrs_status launched() { return hipGetLastError() == hipSuccess ? LRS_OK : LRS_ERR_HIP; }

// Calls f with the truth value as a constant.
template <typename F>
void with_bool(bool v, F &&f)
{
    if (v)
        f(std::true_type{});
    else
        f(std::false_type{});
}

// Calls f with a value of the row type.
template <typename F>
lrs_status with_type(lrs_row_type t, F &&f)
{
    switch (t) {
    case LRS_ROW_F32: return f(float{});
    case LRS_ROW_BF16: return f(bf16{});
    case LRS_ROW_F16: return f(f16{});
    }
    return LRS_ERR_INVALID_ARG;
}

// Nothing that the C++ runtime throws (the sort keeps a small table of its kernels'
// occupancy) leaves the C boundary.
template <typename F>
lrs_status guarded(F &&f)
{
    try {
        return f();
    } catch (...) {
        return LRS_ERR_HIP;
    }
}

// The two-phase temp storage convention: LRS_OK with *temp NULL after a query.
inline lrs_status take_temp(void *d_temp, size_t *temp_bytes, size_t total, char **temp)
{
    *temp = nullptr;
    if (d_temp == nullptr) {
        *temp_bytes = total + (kAlign - 1);
        return LRS_OK;
    }
    const size_t pad = (kAlign - (uintptr_t)d_temp % kAlign) % kAlign;
    if (*temp_bytes < total + pad) return LRS_ERR_TEMP_TOO_SMALL;
    *temp = (char *)d_temp + pad;
    return LRS_OK;
}

// Slots: tokens * slots flat indices, int32.
inline bool slots_ok(int64_t tokens, int64_t slots)
{
    return count_ok(tokens) && count_ok(slots) && (__int128)tokens * slots <= kMaxCount;
}

}  // namespace
