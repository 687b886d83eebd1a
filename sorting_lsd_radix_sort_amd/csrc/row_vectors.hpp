// row_vectors.hpp -- rows of a matrix in 16-byte vectors at any alignment, their
// elements in float32, and how a grid covers them: what the kernels of row_kernels.hpp,
// route_kernels.hpp and beam_kernels.hpp share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace lrs_rows {

constexpr int kWave = 64;
constexpr int kThreads = 256;  // four waves, one row or several per workgroup

typedef __bf16 bf16;
typedef _Float16 f16;

// ------------------------------------------------------------------- vectors
//
// 16 bytes of a row at the alignment of one element: the global loads and stores
// of gfx950 take any address, and neighbouring lanes' bytes stay neighbours, so
// rows that begin off a 16-byte boundary cost a line more per wave, not an
// instruction per element.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);  // elements of one 16-byte vector

typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(2)));

// One vector of a row: the elements from column c, `valid` of them (the last vector of
// a row may be short).  A short one is loaded as the 16 bytes that end with the row,
// `back` elements early, and shifted into place once they are there: no byte beyond
// the row is touched, and the loads of several rows are in flight together.  Only in
// a row shorter than a vector (back 0, valid short) are elements loaded one by one.
struct Col {
    int64_t c;
    int valid, back;
};

template <typename T>
__device__ __forceinline__ Col col_of(int64_t cols, int64_t c)
{
    const int valid = cols - c < kVec<T> ? (int)(cols - c) : kVec<T>;
    return {c, valid, valid > 0 && c >= kVec<T> - valid ? kVec<T> - valid : 0};
}

// Right shift of 16 bytes by a number of elements, zeros shifted in.
template <typename T>
__device__ __forceinline__ u32x4 shift_down(u32x4 r, int elements)
{
    const int bytes = elements * (int)sizeof(T);
    if (bytes & 8) r = u32x4{r[2], r[3], 0u, 0u};
    if (bytes & 4) r = u32x4{r[1], r[2], r[3], 0u};
    if constexpr (sizeof(T) == 2)
        if (bytes & 2)
            r = u32x4{r[0] >> 16 | r[1] << 16, r[1] >> 16 | r[2] << 16, r[2] >> 16 | r[3] << 16, r[3] >> 16};
    return r;
}

// Loads a vector of a row.  NT: past the caches, for rows that are read once and more
// of them than the L2s hold.  settle() puts what was loaded into place: elements
// 0..valid - 1, zeros after them.
template <typename T, bool NT = false>
__device__ __forceinline__ u32x4 issue(const T *row, const Col &col)
{
    if (col.valid + col.back == kVec<T>) {
        const u32x4_any *p = reinterpret_cast<const u32x4_any *>(row + (col.c - col.back));
        if constexpr (NT) return __builtin_nontemporal_load(p);
        return *p;
    }
    u32x4 r = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e)
        if (e < col.valid) {
            if constexpr (sizeof(T) == 4)
                r[e] = reinterpret_cast<const uint32_t *>(row + col.c)[e];
            else
                r[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(row + col.c)[e] << (16 * (e & 1));
        }
    return r;
}

template <typename T>
__device__ __forceinline__ u32x4 settle(u32x4 r, const Col &col)
{
    return col.back > 0 ? shift_down<T>(r, col.back) : r;
}

template <typename T, bool NT = false>
__device__ __forceinline__ u32x4 load_col(const T *row, const Col &col)
{
    return settle<T>(issue<T, NT>(row, col), col);
}

// Stores `valid` elements at p: one store, or one for each bit of a short count.
template <typename T, bool NT = false>
__device__ __forceinline__ void store_raw(T *p, u32x4 r, int valid)
{
    if (valid >= kVec<T>) {
        u32x4_any *q = reinterpret_cast<u32x4_any *>(p);
        if constexpr (NT)
            __builtin_nontemporal_store((u32x4_any)r, q);
        else
            *q = r;
        return;
    }
    if (valid <= 0) return;
    const int words = valid * (int)sizeof(T) / 4;  // whole ones
    char *at = reinterpret_cast<char *>(p);
    if (words & 2) *reinterpret_cast<u32x2_any *>(at) = u32x2_any{r[0], r[1]};
    if (words & 1) *reinterpret_cast<u32_any *>(at + (words & 2) * 4) = words & 2 ? r[2] : r[0];
    if constexpr (sizeof(T) == 2) {
        if (valid & 1) {
            uint32_t q = 0u;
#pragma unroll
            for (int w = 0; w < 4; ++w) q |= w == words ? r[w] : 0u;
            reinterpret_cast<uint16_t *>(at)[valid - 1] = (uint16_t)q;
        }
    }
}

template <typename T, bool NT = false>
__device__ __forceinline__ void store_col(T *row, u32x4 r, const Col &col)
{
    store_raw<T, NT>(row + col.c, r, col.valid);
}

// Element e of a vector in float32 (exact for all three types).
template <typename T>
__device__ __forceinline__ float element(u32x4 r, int e)
{
    if constexpr (sizeof(T) == 4) {
        const uint32_t word = r[e];
        return __builtin_bit_cast(float, word);
    } else if constexpr (__is_same(T, bf16)) {
        return __builtin_bit_cast(float, e & 1 ? r[e / 2] & 0xFFFF0000u : r[e / 2] << 16);
    } else {
        return (float)__builtin_bit_cast(f16, (uint16_t)(r[e / 2] >> (16 * (e & 1))));
    }
}

// The vector with element e replaced.
template <typename T>
__device__ __forceinline__ u32x4 with_element(u32x4 r, int e, float v)
{
    if constexpr (sizeof(T) == 4) {
        r[e] = __builtin_bit_cast(uint32_t, v);
    } else {
        const uint32_t h = __builtin_bit_cast(uint16_t, (T)v);
        r[e / 2] = e & 1 ? (r[e / 2] & 0xFFFFu) | h << 16 : (r[e / 2] & 0xFFFF0000u) | h;
    }
    return r;
}

// float32 values rounded once, to nearest even, to a vector of T.
template <typename T>
__device__ __forceinline__ u32x4 pack(const float (&v)[kVec<T>])
{
    u32x4 r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = __builtin_bit_cast(uint32_t, v[e]);
    } else {
        typedef T pair __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const pair q = {(T)v[2 * e], (T)v[2 * e + 1]};
            r[e] = __builtin_bit_cast(uint32_t, q);
        }
    }
    return r;
}

// A scalar of one of the row types (0 float32, 1 bfloat16, 2 float16: lrs_row_type).
__device__ __forceinline__ float load_scalar(const void *p, int type, int64_t i)
{
    if (type == 0) return ((const float *)p)[i];
    if (type == 1) return (float)((const bf16 *)p)[i];
    return (float)((const f16 *)p)[i];
}

__device__ __forceinline__ void store_scalar(void *p, int type, int64_t i, float v)
{
    if (type == 0)
        ((float *)p)[i] = v;
    else if (type == 1)
        ((bf16 *)p)[i] = (bf16)v;
    else
        ((f16 *)p)[i] = (f16)v;
}

// ---------------------------------------------------------------------- grid
//
// A workgroup serves kThreads / tx rows, tx = 2^tx_log2 lanes each, and tx vectors of
// each row; grid.x runs over a row's pieces and grid.y over the rows, both in strides
// where there are more than kMaxGridX and kMaxGridY.
//
// Kernels take their counts as 32-bit words, work out what follows from them (vectors,
// tiles, the grid itself) and ask for nothing that the runtime passes beside their own
// arguments: a launch with up to 96 bytes of arguments takes 2.8 us of the host's time,
// one with 128 or more 3.5 to 3.9, and a use of gridDim adds 66 bytes and more.  (The
// two that prepare and finish an order by the library's sort do use it, beside the sort's
// own launches.)
constexpr int64_t kMaxGridX = 1 << 20, kMaxGridY = 65535;

// The row that this thread serves in row tile `tile`; the same for a whole wave
// where a wave serves one row, which the compiler is told.
template <bool WAVE_ROW>
__device__ __forceinline__ int64_t row_of(int tx_log2, int64_t tile)
{
    int r = (int)(threadIdx.x >> tx_log2);
    if constexpr (WAVE_ROW) r = __builtin_amdgcn_readfirstlane(r);
    return tile * (kThreads >> tx_log2) + r;
}

template <typename T>
__device__ __forceinline__ int vecs_of(int cols)
{
    return (int)(((uint32_t)cols + kVec<T> - 1) / (uint32_t)kVec<T>);
}

__device__ __forceinline__ int64_t tiles_of(int64_t count, int log2) { return (count + (1 << log2) - 1) >> log2; }

constexpr int kThreadsLog2 = 8;
static_assert(kThreads == 1 << kThreadsLog2, "rows of a tile are found by shifts");

// Calls f(row, vector) for each that this thread serves.  The grid is the number of
// tiles, up to the two limits: so a step of a limit leaves it at once where there are
// no more, and nothing has to be worked out before the first loads.
template <bool WAVE_ROW, typename F>
__device__ __forceinline__ void for_tiles(int tx_log2, int rows, int vecs, F &&f)
{
    int64_t tile = blockIdx.y;
    do {
        const int64_t row = row_of<WAVE_ROW>(tx_log2, tile);
        if (row < rows) {
            int64_t piece = blockIdx.x;
            do {
                const int64_t vec = (piece << tx_log2) + (threadIdx.x & ((1 << tx_log2) - 1));
                if (vec < vecs) f(row, vec);
                piece += kMaxGridX;
            } while (piece << tx_log2 < vecs);
        }
        tile += kMaxGridY;
    } while (tile << (kThreadsLog2 - tx_log2) < rows);
}

}  // namespace lrs_rows
