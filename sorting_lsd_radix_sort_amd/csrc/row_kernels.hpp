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

// The same past the caches (NT): for rows that are read or written once and more of
// them than the L2 holds.
template <bool NT, typename T>
__device__ __forceinline__ u32x4 load_once(const T *p, int valid)
{
    if constexpr (NT)
        if (valid >= kVec<T>) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(p));
    return load_raw<T>(p, valid);
}

template <bool NT, typename T>
__device__ __forceinline__ void store_once(T *p, u32x4 r, int valid)
{
    if constexpr (NT)
        if (valid >= kVec<T>) {
            __builtin_nontemporal_store((u32x4_any)r, reinterpret_cast<u32x4_any *>(p));
            return;
        }
    store_raw<T>(p, r, valid);
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

// A token's rows are summed in the order of its slots, in float32, SLOTS of them in
// flight per lane.
template <typename T, bool WAVE_ROW, int SLOTS, bool NT>
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
        for (int k0 = 0; k0 < slots; k0 += SLOTS) {
            uint32_t p[SLOTS];
            u32x4 r[SLOTS];
            float w[SLOTS];
#pragma unroll
            for (int u = 0; u < SLOTS; ++u) {
                p[u] = k0 + u < slots ? (uint32_t)position[t * slots + k0 + u] : ~0u;
                if (p[u] < num_rows) {
                    r[u] = load_once<NT>(rows + (int64_t)p[u] * ld_rows + c, valid);
                    w[u] = weights != nullptr ? load_scalar(weights, weight_type, t * slots + k0 + u) : 1.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < SLOTS; ++u)
                if (p[u] < num_rows) {
#pragma unroll
                    for (int e = 0; e < kVec<T>; ++e) sum[e] = __builtin_fmaf(w[u], element<T>(r[u], e), sum[e]);
                }
        }
        store_once<NT>(y + t * ld_y + c, pack<T>(sum), valid);
    }
}

// Sum over the lanes of a row: a whole wave (WAVE_ROW) or 2^tx_log2 lanes of it, in
// a fixed order, the same for every lane.
template <bool WAVE_ROW>
__device__ __forceinline__ float lanes_sum(float v, int tx_log2)
{
    if constexpr (WAVE_ROW) {
        auto add = [&](auto ctrl, auto rows) {
            const int other = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl.value, rows.value, 0xf, false);
            v += __builtin_bit_cast(float, other);
        };
        using std::integral_constant;
        add(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});  // row_shr:1
        add(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});  // row_shr:2
        add(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});  // row_shr:4
        add(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});  // row_shr:8
        add(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});  // row_bcast:15
        add(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});  // row_bcast:31
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
    } else {
        for (int x = 1 << tx_log2 >> 1; x >= 1; x >>= 1) v += __shfl_xor(v, x);
        return v;
    }
}

// A row tile serves whole tokens, slot by slot (grid.x of their slots at once): a
// slot's row is read, its inner product with the token's grad_y formed, and its
// gradient stored; grad_y comes from cache after the first slot.  rows and grad_rows
// may be the same memory: a thread reads each element before it stores there.
template <typename T, bool WAVE_ROW, bool NT>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(const T *__restrict__ grad_y, int64_t ld_grad_y,
                                                                const T *rows, int64_t ld_rows, uint32_t num_rows,
                                                                const int32_t *__restrict__ position, int weight_type,
                                                                const void *__restrict__ weights, int64_t tokens,
                                                                int slots, int64_t cols, T *grad_rows,
                                                                int64_t ld_grad_rows, void *__restrict__ grad_weights,
                                                                Tiling tl)
{
    __shared__ float s_part[kThreads / kWave];
    const int lane = threadIdx.x & ((1 << tl.tx_log2) - 1);
    const int waves = 1 << tl.tx_log2 >> 6;  // per token; 0 where a wave serves several
    for (int64_t tile = blockIdx.y; tile < tl.row_tiles; tile += gridDim.y) {
        const int64_t t = row_of<WAVE_ROW>(tl, tile);
        for (int64_t k = blockIdx.x; k < slots; k += gridDim.x) {
            const uint32_t p = t < tokens ? (uint32_t)position[t * slots + k] : ~0u;
            float dot = 0.0f;
            if (p < num_rows) {
                const float w = weights != nullptr ? load_scalar(weights, weight_type, t * slots + k) : 1.0f;
                for (int64_t vec = lane; vec < tl.vecs; vec += 1 << tl.tx_log2) {
                    const int64_t c = vec * kVec<T>;
                    const int valid = valid_of(cols, c, kVec<T>);
                    const u32x4 g = load_raw<T>(grad_y + t * ld_grad_y + c, valid);
                    if (grad_weights != nullptr) {
                        const u32x4 r = load_once<NT>(rows + (int64_t)p * ld_rows + c, valid);
#pragma unroll
                        for (int e = 0; e < kVec<T>; ++e) dot = __builtin_fmaf(element<T>(g, e), element<T>(r, e), dot);
                    }
                    float out[kVec<T>];
#pragma unroll
                    for (int e = 0; e < kVec<T>; ++e) out[e] = w * element<T>(g, e);
                    store_once<NT>(grad_rows + (int64_t)p * ld_grad_rows + c, pack<T>(out), valid);
                }
            }
            if (grad_weights == nullptr) continue;
            dot = lanes_sum<WAVE_ROW>(dot, tl.tx_log2);
            if (waves > 1) {
                __syncthreads();  // (the last slot's parts have been read)
                if ((threadIdx.x & (kWave - 1)) == 0) s_part[threadIdx.x / kWave] = dot;
                __syncthreads();
                if (lane == 0) {
                    dot = 0.0f;
                    for (int v = 0; v < waves; ++v) dot += s_part[threadIdx.x / kWave + v];
                }
            }
            if (lane == 0 && t < tokens) store_scalar(grad_weights, weight_type, t * slots + k, dot);
        }
    }
}

// ----------------------------------------------------------------- embedding

template <typename T, typename ID, bool WAVE_ROW, bool NT>
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
        store_once<NT>(y + i * ld_y + c, r, valid);
    }
}

// The gradient's sums.  The sorted ids are cut into pieces of `piece` slots, one
// piece of a column tile per unit of work, whatever the ids: a run of equal ids may
// be one slot or all of them, and pieces stay equal.  A run inside a piece is summed
// in registers and stored at once.  A run that crosses pieces leaves one float32
// partial sum in each: slot 0 of a piece for a run that began earlier, slot 1 for one
// that begins in it and goes on; embedding_join_kernel adds them up, in order.
struct Pieces {
    int64_t n;        // sorted slots
    int piece;        // slots per piece
    int64_t count;    // pieces
    uint32_t groups;  // ids at or above it are of no row (sorted last)
};

template <typename G, int E>
__device__ __forceinline__ void store_values(G *p, const float (&v)[E], int valid)
{
#pragma unroll
    for (int q = 0; q < E; q += kVec<G>) {
        float part[kVec<G>];
#pragma unroll
        for (int e = 0; e < kVec<G>; ++e) part[e] = v[q + e];
        if (valid > q) store_raw<G>(p + q, pack<G>(part), valid - q);
    }
}

// scale * sum, added to what is there if `accumulate`, rounded once.
template <typename G, int E>
__device__ __forceinline__ void store_grad(G *p, const float (&sum)[E], float scale, int accumulate, int valid)
{
    float v[E];
    if (accumulate) {
#pragma unroll
        for (int q = 0; q < E; q += kVec<G>) {
            const u32x4 old = load_raw<G>(p + q, valid - q);
#pragma unroll
            for (int e = 0; e < kVec<G>; ++e) v[q + e] = __builtin_fmaf(scale, sum[q + e], element<G>(old, e));
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = scale * sum[e];
    }
    store_values<G, E>(p, v, valid);
}

template <typename T, typename G, bool WAVE_ROW>
__device__ void sum_piece(const T *__restrict__ grad_y, int64_t ld_grad_y, const uint32_t *__restrict__ keys,
                          const uint32_t *__restrict__ order, Pieces pc, float scale, G *__restrict__ grad,
                          int64_t ld_grad, int64_t cols, int64_t cols_padded, float *__restrict__ partial,
                          int accumulate, int64_t piece, int64_t vec)
{
    constexpr int E = kVec<T>;
    constexpr int UNROLL = 8;  // rows in flight per lane
    const int64_t c = vec * E;
    const int valid = valid_of(cols, c, E);
    const int64_t lo = piece * pc.piece;
    int64_t hi = lo + pc.piece < pc.n ? lo + pc.piece : pc.n;
    uint32_t run = keys[lo];
    bool here = lo == 0 || keys[lo - 1] != run;  // the run begins in this piece
    float sum[E] = {};
    auto leave = [&](bool goes_on) {
        if (run >= pc.groups) return;
        if (here && !goes_on)
            store_grad<G, E>(grad + (int64_t)run * ld_grad + c, sum, scale, accumulate, valid);
        else  // (padded rows of whole vectors: no partial store)
            store_values<float, E>(partial + (piece * 2 + (here ? 1 : 0)) * cols_padded + c, sum, E);
    };
    for (int64_t j = lo; j < hi && run < pc.groups; j += UNROLL) {
        u32x4 r[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
            if (j + u < hi && keys[j + u] < pc.groups)
                r[u] = load_raw<T>(grad_y + (int64_t)order[j + u] * ld_grad_y + c, valid);
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (j + u < hi) {
                const uint32_t k = keys[j + u];
                if (k != run) {
                    leave(false);
                    run = k;
                    here = true;
#pragma unroll
                    for (int e = 0; e < E; ++e) sum[e] = 0.0f;
                }
                if (k < pc.groups) {
#pragma unroll
                    for (int e = 0; e < E; ++e) sum[e] += element<T>(r[u], e);
                }
            }
        }
    }
    leave(hi < pc.n && keys[hi] == run);
}

// Rows that no id names are zeros.  A workgroup looks kFillRows rows up in the
// sorted ids (one lane each) and stores those that are not there.
constexpr int kFillRows = 32;

template <typename G>
__device__ void fill_rows(const uint32_t *__restrict__ keys, int64_t n, G *__restrict__ grad, int64_t ld_grad,
                          int64_t num_ids, int64_t cols, int64_t tile)
{
    __shared__ int s_named[kFillRows];
    __syncthreads();
    if (threadIdx.x < kFillRows) {
        const int64_t v = tile * kFillRows + threadIdx.x;
        int named = 1;
        if (v < num_ids) {
            const int64_t j = lower_bound(keys, n, (uint32_t)v);
            named = j < n && keys[j] == (uint32_t)v;
        }
        s_named[threadIdx.x] = named;
    }
    __syncthreads();
    const u32x4 zero = {0u, 0u, 0u, 0u};
    for (int q = 0; q < kFillRows; ++q) {
        if (s_named[q]) continue;
        G *row = grad + (tile * kFillRows + q) * ld_grad;
        for (int64_t c = (int64_t)threadIdx.x * kVec<G>; c < cols; c += kThreads * kVec<G>)
            store_raw<G>(row + c, zero, valid_of(cols, c, kVec<G>));
    }
}

// The first `sum_blocks` workgroups sum pieces, the others write the empty rows.
template <typename T, typename G, bool WAVE_ROW>
__global__ __launch_bounds__(kThreads) void embedding_grad_kernel(const T *__restrict__ grad_y, int64_t ld_grad_y,
                                                                  const uint32_t *__restrict__ keys,
                                                                  const uint32_t *__restrict__ order, Pieces pc,
                                                                  float scale, G *__restrict__ grad, int64_t ld_grad,
                                                                  int64_t num_ids, int64_t cols, int64_t cols_padded,
                                                                  float *__restrict__ partial, int accumulate,
                                                                  uint32_t sum_blocks, Tiling tl)
{
    if (blockIdx.x < sum_blocks) {
        const int64_t units = tl.row_tiles * tl.col_tiles;
        for (int64_t unit = blockIdx.x; unit < units; unit += sum_blocks) {
            const int64_t piece = row_of<WAVE_ROW>(tl, unit / tl.col_tiles);
            const int64_t vec = ((unit % tl.col_tiles) << tl.tx_log2) + (threadIdx.x & ((1 << tl.tx_log2) - 1));
            if (piece < pc.count && vec < tl.vecs)
                sum_piece<T, G, WAVE_ROW>(grad_y, ld_grad_y, keys, order, pc, scale, grad, ld_grad, cols, cols_padded,
                                          partial, accumulate, piece, vec);
        }
    } else {
        const int64_t tiles = (num_ids + kFillRows - 1) / kFillRows;
        for (int64_t t = blockIdx.x - sum_blocks; t < tiles; t += gridDim.x - sum_blocks)
            fill_rows<G>(keys, pc.n, grad, ld_grad, num_ids, cols, t);
    }
}

// Adds the partial sums of each run that crosses pieces: the workgroup of the piece
// in which the run begins takes that piece's partial and those of the pieces after
// it, four waves a quarter of them each, their sums joined in order.  64 vectors of
// four columns per workgroup.
template <typename G>
__global__ __launch_bounds__(kThreads) void embedding_join_kernel(const uint32_t *__restrict__ keys, Pieces pc,
                                                                  float scale, G *__restrict__ grad, int64_t ld_grad,
                                                                  int64_t cols, int64_t cols_padded,
                                                                  const float *__restrict__ partial, int accumulate,
                                                                  int64_t col_tiles)
{
    constexpr int SLICES = kThreads / kWave;
    __shared__ float s_sum[SLICES][kWave][4];
    const int64_t units = (pc.count - 1) * col_tiles;
    const int lane = threadIdx.x & (kWave - 1), slice = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t piece = unit / col_tiles;
        const int64_t lo = piece * pc.piece, hi = lo + pc.piece;  // (the last piece is not among them)
        const uint32_t run = keys[hi - 1];
        if (run >= pc.groups || keys[hi] != run || (keys[lo] == run && lo > 0 && keys[lo - 1] == run)) continue;
        // the run's last slot, then its last piece
        int64_t a = hi, b = pc.n;  // keys[a] == run; b: past the end
        while (b - a > 1) {
            const int64_t mid = (a + b) >> 1;
            if (keys[mid] == run)
                a = mid;
            else
                b = mid;
        }
        const int64_t last = a / pc.piece, more = last - piece;  // pieces after the first
        const int64_t per = (more + SLICES - 1) / SLICES;
        const int64_t from = piece + 1 + slice * per, to = from + per < last + 1 ? from + per : last + 1;
        const int64_t c = ((unit % col_tiles) * kWave + lane) * 4;
        float sum[4] = {};
        if (c < cols) {
            if (slice == 0) {
                const u32x4 r = load_raw<float>(partial + (piece * 2 + 1) * cols_padded + c, 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] = element<float>(r, e);
            }
#pragma unroll 8
            for (int64_t p = from; p < to; ++p) {
                const u32x4 r = load_raw<float>(partial + p * 2 * cols_padded + c, 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += element<float>(r, e);
            }
        }
        if (more > 1) {  // else the first wave has it all
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 4; ++e) s_sum[slice][lane][e] = sum[e];
            __syncthreads();
            if (slice == 0) {
                for (int w = 1; w < SLICES; ++w)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[e] += s_sum[w][lane][e];
            }
        }
        if (slice == 0 && c < cols) {
            const int valid = valid_of(cols, c, 4);
            G *p = grad + (int64_t)run * ld_grad + c;
            // (four columns are half a vector of 16-bit elements: element by element)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < valid) p[e] = (G)(accumulate ? __builtin_fmaf(scale, sum[e], (float)p[e]) : scale * sum[e]);
        }
    }
}

}  // namespace lrs_rows
