// row_kernels.hpp -- gfx950 (CDNA4, wave64) kernels that move and sum the rows of
// a matrix in the order of small integer keys (include/lrsort_rows.h).
//
// All of them are bound by memory: a row element is read once, takes part in at
// most a few operations, and is written once.  So each lane moves 16 bytes at a
// time, neighbouring lanes neighbouring bytes of one row, and a row's index (its
// position, id or run) is formed once per wave where a wave serves a single row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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

// `valid` elements (at most a vector's) from p; the others are zero.
template <typename T>
__device__ __forceinline__ u32x4 load_raw(const T *p, int valid)
{
    if (valid >= kVec<T>) return *reinterpret_cast<const u32x4_any *>(p);
    u32x4 r = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) {
        if (e < valid) {
            if constexpr (sizeof(T) == 4)
                r[e] = reinterpret_cast<const uint32_t *>(p)[e];
            else
                r[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[e] << (16 * (e & 1));
        }
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void store_raw(T *p, u32x4 r, int valid)
{
    if (valid >= kVec<T>) {
        *reinterpret_cast<u32x4_any *>(p) = r;
        return;
    }
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) {
        if (e < valid) {
            if constexpr (sizeof(T) == 4)
                reinterpret_cast<uint32_t *>(p)[e] = r[e];
            else
                reinterpret_cast<uint16_t *>(p)[e] = (uint16_t)(r[e / 2] >> (16 * (e & 1)));
        }
    }
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
// A workgroup serves kThreads / tx rows, tx lanes each (a power of two), and tx
// vectors of each row; grid.x runs over a row's pieces and grid.y over the rows,
// both in strides where there are more than the grid holds.
struct Tiling {
    int tx_log2;
    int64_t vecs;  // vectors per row, the last perhaps short
    int64_t row_tiles;
    int64_t col_tiles;
};

// The row that this thread serves in row tile `tile`; the same for a whole wave
// where a wave serves one row, which the compiler is told.
template <bool WAVE_ROW>
__device__ __forceinline__ int64_t row_of(const Tiling &tl, int64_t tile)
{
    const int ty = kThreads >> tl.tx_log2;
    int r = (int)(threadIdx.x >> tl.tx_log2);
    if constexpr (WAVE_ROW) r = __builtin_amdgcn_readfirstlane(r);
    return tile * ty + r;
}

#define LRS_FOR_TILES(tl, rows, row, vec)                                                              \
    for (int64_t tile_ = blockIdx.y; tile_ < (tl).row_tiles; tile_ += gridDim.y)                       \
        if (const int64_t row = row_of<WAVE_ROW>(tl, tile_); row < (rows))                             \
            for (int64_t ct_ = blockIdx.x; ct_ < (tl).col_tiles; ct_ += gridDim.x)                     \
                if (const int64_t vec = (ct_ << (tl).tx_log2) + (threadIdx.x & ((1 << (tl).tx_log2) - 1)); \
                    vec < (tl).vecs)

__device__ __forceinline__ int valid_of(int64_t cols, int64_t c, int vec)
{
    return cols - c < vec ? (int)(cols - c) : vec;
}

// ------------------------------------------------------------------ grouping

// Keys of the grouping sort: id - first where that is below `groups`, else
// `groups` (sorted last), and the indices that travel with them.
template <typename ID>
__global__ __launch_bounds__(kThreads) void group_keys_kernel(const ID *__restrict__ ids, int64_t n, int64_t first,
                                                              uint32_t groups, uint32_t *__restrict__ keys,
                                                              uint32_t *__restrict__ index)
{
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const uint64_t g = (uint64_t)ids[i] - (uint64_t)first;
        keys[i] = g < groups ? (uint32_t)g : groups;
        index[i] = (uint32_t)i;
    }
}

// First j with keys[j] >= g (keys ascending).
__device__ __forceinline__ int64_t lower_bound(const uint32_t *__restrict__ keys, int64_t n, uint32_t g)
{
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (keys[mid] < g)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// From the sorted keys and their indices: each index's position, and where each
// group begins.
__global__ __launch_bounds__(kThreads) void group_finish_kernel(const uint32_t *__restrict__ keys,
                                                                const uint32_t *__restrict__ order, int64_t n,
                                                                uint32_t groups, int32_t *__restrict__ position,
                                                                int32_t *__restrict__ offsets)
{
    const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x, stride = (int64_t)gridDim.x * kThreads;
    if (position != nullptr)
        for (int64_t j = first; j < n; j += stride) position[order[j]] = keys[j] < groups ? (int32_t)j : -1;
    if (offsets != nullptr)
        for (int64_t g = first; g <= (int64_t)groups; g += stride) offsets[g] = (int32_t)lower_bound(keys, n, (uint32_t)g);
}

// ------------------------------------------------------- rows to their places

// A token's row is read once and stored `slots` times: the bytes of the rows
// written and of x, nothing else.  T: an unsigned word of the element's size.
template <typename T, bool WAVE_ROW>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(const T *__restrict__ x, int64_t ld_x,
                                                            const int32_t *__restrict__ position, int64_t tokens,
                                                            int slots, int64_t cols, T *__restrict__ rows,
                                                            int64_t ld_rows, uint32_t num_rows, Tiling tl)
{
    LRS_FOR_TILES(tl, tokens, t, vec)
    {
        const int64_t c = vec * kVec<T>;
        const int valid = valid_of(cols, c, kVec<T>);
        const u32x4 v = load_raw<T>(x + t * ld_x + c, valid);
        for (int k = 0; k < slots; ++k) {
            const uint32_t p = (uint32_t)position[t * slots + k];
            if (p < num_rows) store_raw<T>(rows + (int64_t)p * ld_rows + c, v, valid);
        }
    }
}

// A token's rows are summed in the order of its slots, in float32.
template <typename T, bool WAVE_ROW>
__global__ __launch_bounds__(kThreads) void combine_kernel(const T *__restrict__ rows, int64_t ld_rows,
                                                           uint32_t num_rows, const int32_t *__restrict__ position,
                                                           int weight_type, const void *__restrict__ weights,
                                                           int64_t tokens, int slots, int64_t cols,
                                                           T *__restrict__ y, int64_t ld_y, Tiling tl)
{
    LRS_FOR_TILES(tl, tokens, t, vec)
    {
        const int64_t c = vec * kVec<T>;
        const int valid = valid_of(cols, c, kVec<T>);
        float sum[kVec<T>] = {};
        for (int k = 0; k < slots; ++k) {
            const uint32_t p = (uint32_t)position[t * slots + k];
            if (p >= num_rows) continue;
            const u32x4 r = load_raw<T>(rows + (int64_t)p * ld_rows + c, valid);
            const float w = weights != nullptr ? load_scalar(weights, weight_type, t * slots + k) : 1.0f;
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e) sum[e] = __builtin_fmaf(w, element<T>(r, e), sum[e]);
        }
        store_raw<T>(y + t * ld_y + c, pack<T>(sum), valid);
    }
}

// Sum over the workgroup, in a fixed order; every thread calls it.
__device__ __forceinline__ float block_sum(float v, float *s_part)
{
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1) v += __shfl_xor(v, x);
    __syncthreads();
    if ((threadIdx.x & (kWave - 1)) == 0) s_part[threadIdx.x / kWave] = v;
    __syncthreads();
    float all = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) all += s_part[w];
    return all;
}

// One workgroup per slot: its row of grad_rows is w times the token's grad_y, and
// the weight's gradient their inner product.  rows and grad_rows may be the same
// memory: a thread reads each element before it stores there.
template <typename T>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(const T *__restrict__ grad_y, int64_t ld_grad_y,
                                                                const T *rows, int64_t ld_rows, uint32_t num_rows,
                                                                const int32_t *__restrict__ position, int weight_type,
                                                                const void *__restrict__ weights, int64_t n, int slots,
                                                                int64_t cols, T *grad_rows, int64_t ld_grad_rows,
                                                                void *__restrict__ grad_weights)
{
    __shared__ float s_part[kThreads / kWave];
    const int64_t vecs = (cols + kVec<T> - 1) / kVec<T>;
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
        const uint32_t p = (uint32_t)position[i];
        const bool there = p < num_rows;
        float dot = 0.0f;
        if (there) {
            const float w = weights != nullptr ? load_scalar(weights, weight_type, i) : 1.0f;
            for (int64_t vec = threadIdx.x; vec < vecs; vec += kThreads) {
                const int64_t c = vec * kVec<T>;
                const int valid = valid_of(cols, c, kVec<T>);
                const u32x4 g = load_raw<T>(grad_y + i / slots * ld_grad_y + c, valid);
                if (grad_weights != nullptr) {
                    const u32x4 r = load_raw<T>(rows + (int64_t)p * ld_rows + c, valid);
#pragma unroll
                    for (int e = 0; e < kVec<T>; ++e) dot = __builtin_fmaf(element<T>(g, e), element<T>(r, e), dot);
                }
                float out[kVec<T>];
#pragma unroll
                for (int e = 0; e < kVec<T>; ++e) out[e] = w * element<T>(g, e);
                store_raw<T>(grad_rows + (int64_t)p * ld_grad_rows + c, pack<T>(out), valid);
            }
        }
        if (grad_weights != nullptr) {
            dot = block_sum(dot, s_part);
            if (threadIdx.x == 0) store_scalar(grad_weights, weight_type, i, dot);
        }
    }
}

// ----------------------------------------------------------------- embedding

template <typename T, typename ID, bool WAVE_ROW>
__global__ __launch_bounds__(kThreads) void embedding_kernel(const T *__restrict__ table, int64_t ld_table,
                                                             uint32_t num_ids, const ID *__restrict__ ids, int64_t n,
                                                             int64_t first, float scale, int64_t cols,
                                                             T *__restrict__ y, int64_t ld_y, Tiling tl)
{
    LRS_FOR_TILES(tl, n, i, vec)
    {
        const int64_t c = vec * kVec<T>;
        const int valid = valid_of(cols, c, kVec<T>);
        const uint64_t v = (uint64_t)ids[i] - (uint64_t)first;
        u32x4 r = {0u, 0u, 0u, 0u};
        if (v < num_ids) {
            r = load_raw<T>(table + (int64_t)v * ld_table + c, valid);
            if (scale != 1.0f) {
                float out[kVec<T>];
#pragma unroll
                for (int e = 0; e < kVec<T>; ++e) out[e] = scale * element<T>(r, e);
                r = pack<T>(out);
            }
        }
        store_raw<T>(y + i * ld_y + c, r, valid);
    }
}

// One row of the table's gradient per row of the grid: the run of its id in the
// sorted keys is found by bisection and its rows are summed in order.
template <typename T, typename G, bool WAVE_ROW>
__global__ __launch_bounds__(kThreads) void embedding_grad_kernel(const T *__restrict__ grad_y, int64_t ld_grad_y,
                                                                  const uint32_t *__restrict__ keys,
                                                                  const uint32_t *__restrict__ order, int64_t n,
                                                                  float scale, G *__restrict__ grad, int64_t ld_grad,
                                                                  int64_t num_ids, int64_t cols, int accumulate,
                                                                  Tiling tl)
{
    LRS_FOR_TILES(tl, num_ids, v, vec)
    {
        const int64_t c = vec * kVec<G>;
        const int valid = valid_of(cols, c, kVec<G>);
        int64_t j = lower_bound(keys, n, (uint32_t)v);
        const bool any = j < n && keys[j] == (uint32_t)v;
        if (accumulate && !any) continue;
        float sum[kVec<G>] = {};
        for (; j < n && keys[j] == (uint32_t)v; ++j) {
            const T *src = grad_y + (int64_t)order[j] * ld_grad_y + c;
#pragma unroll
            for (int e = 0; e < kVec<G>; ++e)
                if (e < valid) sum[e] += (float)src[e];
        }
        if (accumulate) {
            const u32x4 old = load_raw<G>(grad + v * ld_grad + c, valid);
#pragma unroll
            for (int e = 0; e < kVec<G>; ++e) sum[e] = __builtin_fmaf(scale, sum[e], element<G>(old, e));
        } else {
#pragma unroll
            for (int e = 0; e < kVec<G>; ++e) sum[e] *= scale;
        }
        store_raw<G>(grad + v * ld_grad + c, pack<G>(sum), valid);
    }
}

}  // namespace lrs_rows
