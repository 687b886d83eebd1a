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

#include "row_vectors.hpp"

namespace lrs_rows {

// ------------------------------------------------------------------ grouping

// Keys of the grouping sort: id - first where that is below `groups`, else
// `groups` (sorted last), and the indices that travel with them.  `clear`, where
// given, is a word that the first kernel of an order sets to zero for a later one.
template <typename ID>
__global__ __launch_bounds__(kThreads) void group_keys_kernel(const ID *__restrict__ ids, int n, int64_t first,
                                                              uint32_t groups, uint32_t *__restrict__ keys,
                                                              uint32_t *__restrict__ index, uint32_t *clear)
{
    if (clear != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *clear = 0;
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
        for (int64_t g = first; g <= (int64_t)groups; g += stride)
            offsets[g] = (int32_t)lower_bound(keys, n, (uint32_t)g);
}

// ------------------------------------------------------- rows to their places

// A token's row is read once and stored `slots` times: the bytes of the rows
// written and of x, nothing else (reading x once per row written, in the rows' order,
// took 293 us instead of 245 at 16,384 tokens x 8 x 4096 bf16).  One vector a thread:
// with two, four times as much is being written at once, and it took 333.  Bound by
// HBM: 225 us for 1.21 GB, 5.4 TB/s, where rows in sequence would take 213 and a fill
// of the same bytes 157.  A token's row is read also where none of its slots has a
// position.  T: an unsigned word of the element's size.
template <typename T, bool WAVE_ROW>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(const T *__restrict__ x, int64_t ld_x,
                                                            const int32_t *__restrict__ position, int tokens,
                                                            int slots, int cols, uint32_t num_rows,
                                                            T *__restrict__ rows, int64_t ld_rows, int tx_log2)
{
    for_tiles<WAVE_ROW>(tx_log2, tokens, vecs_of<T>(cols), [&](int64_t t, int64_t vec) {
        const Col col = col_of<T>(cols, vec * kVec<T>);
        const u32x4 v = load_col<T>(x + t * ld_x, col);
        for (int k = 0; k < slots; ++k) {
            const uint32_t p = (uint32_t)position[t * slots + k];
            if (p < num_rows) store_col<T>(rows + (int64_t)p * ld_rows, v, col);
        }
    });
}

// A token's rows are summed in the order of its slots, in float32, SLOTS of them in
// flight per lane.  Bound by HBM: 16,384 tokens x 8 x 4096 bf16 in 200 us, 1.21 GB at
// 6.0 TB/s (a read of as much reaches 7.1), calls back to back with one slot in flight
// (two take 11 us more, eight 17); right behind their gradient, whose stores the caches
// still hold, 213.  Rows in sequence would take 190.
template <typename T, bool WAVE_ROW, int SLOTS, bool NT>
__global__ __launch_bounds__(kThreads) void combine_kernel(const T *__restrict__ rows, int64_t ld_rows,
                                                           uint32_t num_rows, int weight_type,
                                                           const int32_t *__restrict__ position,
                                                           const void *__restrict__ weights, int tokens, int slots,
                                                           int cols, int tx_log2, T *__restrict__ y, int64_t ld_y)
{
    for_tiles<WAVE_ROW>(tx_log2, tokens, vecs_of<T>(cols), [&](int64_t t, int64_t vec) {
        const Col col = col_of<T>(cols, vec * kVec<T>);
        float sum[kVec<T>] = {};
        for (int k0 = 0; k0 < slots; k0 += SLOTS) {
            uint32_t p[SLOTS];
            u32x4 r[SLOTS];
            float w[SLOTS];
#pragma unroll
            for (int u = 0; u < SLOTS; ++u) {
                p[u] = k0 + u < slots ? (uint32_t)position[t * slots + k0 + u] : ~0u;
                if (p[u] < num_rows) {
                    r[u] = issue<T, NT>(rows + (int64_t)p[u] * ld_rows, col);
                    w[u] = weights != nullptr ? load_scalar(weights, weight_type, t * slots + k0 + u) : 1.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < SLOTS; ++u)
                if (p[u] < num_rows) {
                    const u32x4 v = settle<T>(r[u], col);
#pragma unroll
                    for (int e = 0; e < kVec<T>; ++e) sum[e] = __builtin_fmaf(w[u], element<T>(v, e), sum[e]);
                }
        }
        store_col<T, NT>(y + t * ld_y, pack<T>(sum), col);
    });
}

// Sum over the lanes of a row: a whole wave (WAVE_ROW) or 2^tx_log2 lanes of it, in
// a fixed order, the same for every lane.
template <bool WAVE_ROW>
__device__ __forceinline__ float lanes_sum(float v, int tx_log2)
{
    if constexpr (WAVE_ROW) {
        auto add = [&](auto ctrl, auto rows) {
            const int other =
                __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl.value, rows.value, 0xf, false);
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

// A row tile serves whole tokens, slot by slot (or, where tokens are `few`, every slot
// by a workgroup of its own): a slot's row is read, its inner product with the token's
// grad_y formed, and its gradient stored; grad_y comes from cache after the first
// slot.  rows and grad_rows may be the same memory: a thread reads each element before
// it stores there (a row's last vector also loads elements of the one before it, which
// may be stored meanwhile, and shifts them out).  Bound
// by HBM: 16,384 tokens x 8 x 4096 bf16 in 442 us, 2.28 GB at 5.15 TB/s (calls back to
// back; 430 behind a sum of rows); a copy reaches 5.9, and the same rows in sequence 395
// to 413 us.  Slots two or eight at a time took 447 and 469, a wave per token (no
// barrier) 478, a workgroup per slot 465.
template <typename T, bool WAVE_ROW, bool NT>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(const T *__restrict__ grad_y, int64_t ld_grad_y,
                                                                const T *rows, int64_t ld_rows,
                                                                const int32_t *__restrict__ position,
                                                                const void *__restrict__ weights, T *grad_rows,
                                                                int64_t ld_grad_rows, void *__restrict__ grad_weights,
                                                                uint32_t num_rows, int tokens, int slots, int cols,
                                                                int8_t weight_type, int8_t tx_log2, int16_t few)
{
    __shared__ float s_part[kThreads / kWave];
    const int lane = threadIdx.x & ((1 << tx_log2) - 1);
    const int waves = 1 << tx_log2 >> 6;  // per token; 0 where a wave serves several
    const int vecs = vecs_of<T>(cols);
    const int64_t tiles = tiles_of(tokens, kThreadsLog2 - tx_log2), at_once = few ? kMaxGridX : 1;
    for (int64_t tile = blockIdx.y; tile < tiles; tile += kMaxGridY) {
        const int64_t t = row_of<WAVE_ROW>(tx_log2, tile);
        for (int64_t k = blockIdx.x; k < slots; k += at_once) {
            const uint32_t p = t < tokens ? (uint32_t)position[t * slots + k] : ~0u;
            float dot = 0.0f;
            if (p < num_rows) {
                const float w = weights != nullptr ? load_scalar(weights, weight_type, t * slots + k) : 1.0f;
                for (int64_t vec = lane; vec < vecs; vec += 1 << tx_log2) {
                    const Col col = col_of<T>(cols, vec * kVec<T>);
                    u32x4 g = issue<T>(grad_y + t * ld_grad_y, col);
                    u32x4 r = {0u, 0u, 0u, 0u};
                    if (grad_weights != nullptr) r = issue<T, NT>(rows + (int64_t)p * ld_rows, col);
                    g = settle<T>(g, col);
                    r = settle<T>(r, col);
                    float out[kVec<T>];
#pragma unroll
                    for (int e = 0; e < kVec<T>; ++e) {
                        dot = __builtin_fmaf(element<T>(g, e), element<T>(r, e), dot);
                        out[e] = w * element<T>(g, e);
                    }
                    store_col<T, NT>(grad_rows + (int64_t)p * ld_grad_rows, pack<T>(out), col);
                }
            }
            if (grad_weights == nullptr) continue;
            dot = lanes_sum<WAVE_ROW>(dot, tx_log2);
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

// One vector a thread.  Stores go past the caches where there are many, so that they
// do not displace the table's frequent rows: 32,768 tokens x 5120 bf16 in 63 us
// instead of 110 (the table's rows that occur are read once, 0.4 GB in all).
template <typename T, typename ID, bool WAVE_ROW, bool NT>
__global__ __launch_bounds__(kThreads) void embedding_kernel(const T *__restrict__ table, int64_t ld_table,
                                                             const ID *__restrict__ ids, int64_t first,
                                                             uint32_t num_ids, int n, int cols, float scale,
                                                             T *__restrict__ y, int64_t ld_y, int tx_log2)
{
    for_tiles<WAVE_ROW>(tx_log2, n, vecs_of<T>(cols), [&](int64_t i, int64_t vec) {
        const Col col = col_of<T>(cols, vec * kVec<T>);
        const uint64_t v = (uint64_t)ids[i] - (uint64_t)first;
        u32x4 r = {0u, 0u, 0u, 0u};
        if (v < num_ids) {
            r = load_col<T>(table + (int64_t)v * ld_table, col);
            if (scale != 1.0f) {
                float out[kVec<T>];
#pragma unroll
                for (int e = 0; e < kVec<T>; ++e) out[e] = scale * element<T>(r, e);
                r = pack<T>(out);
            }
        }
        store_col<T, NT>(y + i * ld_y, r, col);
    });
}

// The gradient's sums, bound by HBM: 65,536 ids x 4096 bf16 of 131,072 rows take 309 us
// here for 1.6 GB (5.3 TB/s), after 26 us of ordering and before 13 of joining.  Sums
// and empty rows in separate phases of one launch: mixed evenly they took 25 us more.
//
// The sorted ids are cut into pieces of `piece` slots, one piece of a column tile per
// unit of work, whatever the ids: a run of equal ids may be one slot or all of them,
// and no unit sums more than two pieces' slots.  A run is summed in registers and stored
// at once by the piece in which it begins, also where it goes on into the next one
// (which passes over it).  Only a run that goes on
// beyond that is left as float32 partial sums, one for each piece that it touches:
// slot 1 of the piece in which it begins, slot 0 of those after it.  The piece in
// which it begins also enters itself in a list (in any order: each run is joined by
// itself), and embedding_join_kernel adds the run's sums up, in order.
constexpr int kKeyPad = 16;

struct Pieces {
    const uint32_t *__restrict__ keys;   // sorted, and the indices that travelled with them
    const uint32_t *__restrict__ order;
    float *__restrict__ partial;  // two rows of whole vectors per piece
    uint32_t *list;               // its length (0 before), then the pieces in which a long run begins
    int n, piece;                 // sorted slots, and slots per piece
    uint32_t groups;              // ids at or above it are of no row (sorted last)
    int cols;
    __device__ __forceinline__ int64_t count() const { return ((int64_t)n + piece - 1) / piece; }
};

// Where the sums go: scale * sum, added to what is there if `accumulate`, rounded once.
template <typename G>
struct GradOut {
    G *grad;
    int64_t ld;
    float scale;
    int accumulate;
};

template <typename G, int E>
__device__ __forceinline__ void store_values(G *p, const float (&v)[E], int valid)
{
#pragma unroll
    for (int q = 0; q < E; q += kVec<G>) {
        float part[kVec<G>];
#pragma unroll
        for (int e = 0; e < kVec<G>; ++e) part[e] = v[q + e];
        store_raw<G>(p + q, pack<G>(part), valid - q);
    }
}

// A vector of a run's sums to its row: one vector of G, or two.
template <typename G, int E>
__device__ __forceinline__ void store_grad(const GradOut<G> &out, uint32_t run, const float (&sum)[E], int cols,
                                           const Col &col)
{
    G *row = out.grad + (int64_t)run * out.ld;
    const float scale = out.scale;
    float v[E];
    if (out.accumulate) {
        u32x4 old[E / kVec<G>];
#pragma unroll
        for (int q = 0; q < E / kVec<G>; ++q) old[q] = issue<G>(row, col_of<G>(cols, col.c + q * kVec<G>));
#pragma unroll
        for (int q = 0; q < E / kVec<G>; ++q) {
            const u32x4 r = settle<G>(old[q], col_of<G>(cols, col.c + q * kVec<G>));
#pragma unroll
            for (int e = 0; e < kVec<G>; ++e)
                v[q * kVec<G> + e] = __builtin_fmaf(scale, sum[q * kVec<G> + e], element<G>(r, e));
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = scale * sum[e];
    }
    store_values<G, E>(row + col.c, v, col.valid);
}

template <typename T, typename G, bool NT>
__device__ __forceinline__ void sum_piece(const T *__restrict__ grad_y, int64_t ld_grad_y, const Pieces &pc,
                                          const GradOut<G> &out, int64_t piece, int64_t vec)
{
    constexpr int E = kVec<T>;
    constexpr int UNROLL = 8;  // rows in flight per lane (4: 16,384 x 2048 added in 75 us instead of 69)
    const uint32_t *__restrict__ keys = pc.keys, *__restrict__ order = pc.order;
    const int cols = pc.cols;
    const int64_t cols_padded = (int64_t)vecs_of<T>(cols) * E;
    const Col col = col_of<T>(cols, vec * E);
    const int64_t lo = piece * pc.piece;
    const int64_t hi = lo + pc.piece < pc.n ? lo + pc.piece : pc.n;
    uint32_t run = keys[lo];
    bool here = lo == 0 || keys[lo - 1] != run;  // the run begins in this piece
    // It began in the piece before and ends in this one, or with it: passed over.
    bool passed = !here && (lo == pc.piece || keys[lo - pc.piece - 1] != run) && (hi == pc.n || keys[hi] != run);
    // The piece's last run is its own to the end if it began here and ends in the next.
    const uint32_t last = keys[hi - 1];
    int64_t more = hi;
    bool goes_on = false;
    if (hi < pc.n && keys[hi] == last) {
        const int64_t next = hi + pc.piece < pc.n ? hi + pc.piece : pc.n;
        goes_on = (lo > 0 && keys[lo - 1] == last) || (next < pc.n && keys[next] == last);
        if (!goes_on) more = next;
    }
    float sum[E] = {};
    auto leave = [&](bool partly) {
        if (run >= pc.groups || passed) return;
        if (here && !partly)
            store_grad<G, E>(out, run, sum, cols, col);
        else  // (padded rows of whole vectors: no partial store)
            store_values<float, E>(pc.partial + (piece * 2 + (here ? 1 : 0)) * cols_padded + col.c, sum, E);
    };
    bool on = true;
    for (int64_t j = lo; on; j += UNROLL) {
        // (keys and order have kKeyPad words more than the slots)
        uint32_t key[UNROLL], at[UNROLL];
        u32x4 r[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) key[u] = keys[j + u], at[u] = order[j + u];
        bool of[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            on = on && key[u] < pc.groups && (j + u < hi || (j + u < more && key[u] == last));
            of[u] = on;
            if (on && !(passed && key[u] == run)) r[u] = issue<T, NT>(grad_y + (int64_t)at[u] * ld_grad_y, col);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (of[u]) {
                if (key[u] != run) {
                    leave(false);
                    run = key[u];
                    here = true;
                    passed = false;
#pragma unroll
                    for (int e = 0; e < E; ++e) sum[e] = 0.0f;
                }
                if (!passed) {
                    const u32x4 v = settle<T>(r[u], col);
#pragma unroll
                    for (int e = 0; e < E; ++e) sum[e] += element<T>(v, e);
                }
            }
        }
    }
    // (ids of no row may follow the last run summed, and be a long run themselves)
    goes_on = goes_on && run == last && run < pc.groups;
    leave(goes_on);
    if (goes_on && here && vec == 0) pc.list[1 + atomicAdd(pc.list, 1u)] = (uint32_t)piece;
}

// First j with keys[j] >= g, by a whole wave: 64 probes a step.
__device__ __forceinline__ int64_t wave_lower_bound(const uint32_t *__restrict__ keys, int64_t n, uint32_t g)
{
    const int lane = threadIdx.x & (kWave - 1);
    int64_t lo = 0, hi = n;  // keys[lo - 1] < g <= keys[hi]
    while (lo < hi) {
        const int64_t step = (hi - lo + kWave - 1) / kWave, at = lo + (lane + 1) * step - 1;
        const int below = __popcll(__ballot(at < hi && keys[at] < g));  // the first `below` probes
        lo += below * step;
        hi = lo + step - 1 < hi ? lo + step - 1 : hi;
    }
    return lo;
}

// Rows that no id names are zeros.  A workgroup looks kFillRows rows up in the
// sorted ids and stores those that are not there: two waves find where the first and
// the row past the last belong, and a lane per row looks between.
constexpr int kFillRows = 16;

template <typename G>
__device__ __forceinline__ void fill_rows(const Pieces &pc, const GradOut<G> &out, int64_t tile, int tx_log2)
{
    const uint32_t *__restrict__ keys = pc.keys;
    const int64_t n = pc.n, num_ids = pc.groups;
    __shared__ int64_t s_range[2];
    __shared__ int s_named[kFillRows];
    __syncthreads();
    if (threadIdx.x < 2 * kWave) {
        const int end = threadIdx.x / kWave;
        const int64_t v = (tile + end) * kFillRows;
        const int64_t j = wave_lower_bound(keys, n, (uint32_t)(v < num_ids ? v : num_ids));
        if ((threadIdx.x & (kWave - 1)) == 0) s_range[end] = j;
    }
    __syncthreads();
    if (threadIdx.x < kFillRows) {
        const int64_t v = tile * kFillRows + threadIdx.x;
        int named = 1;
        if (v < num_ids) {
            int64_t lo = s_range[0], hi = s_range[1];
            const int64_t end = hi;
            while (lo < hi) {
                const int64_t mid = (lo + hi) >> 1;
                if (keys[mid] < (uint32_t)v)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            named = lo < end && keys[lo] == (uint32_t)v;
        }
        s_named[threadIdx.x] = named;
    }
    __syncthreads();
    const u32x4 zero = {0u, 0u, 0u, 0u};
    const int rows_at_once = kThreads >> tx_log2, lane = threadIdx.x & ((1 << tx_log2) - 1);
    const int vecs = vecs_of<G>(pc.cols);
    for (int q = threadIdx.x >> tx_log2; q < kFillRows; q += rows_at_once) {
        if (s_named[q]) continue;
        G *row = out.grad + (tile * kFillRows + q) * out.ld;
        for (int64_t vec = lane; vec < vecs; vec += 1 << tx_log2)
            store_col<G>(row, zero, col_of<G>(pc.cols, vec * kVec<G>));
    }
}

// The first `sum_blocks` workgroups sum pieces, the others write the empty rows.
template <typename T, typename G, bool WAVE_ROW, bool NT>
__global__ __launch_bounds__(kThreads) void embedding_grad_kernel(const T *__restrict__ grad_y, int64_t ld_grad_y,
                                                                  Pieces pc, GradOut<G> out, uint32_t sum_blocks,
                                                                  int16_t tx_log2, int16_t fill_tx_log2)
{
    if (blockIdx.x < sum_blocks) {
        const int vecs = vecs_of<T>(pc.cols);
        const int64_t count = pc.count(), col_tiles = tiles_of(vecs, tx_log2);
        const int64_t units = tiles_of(count, kThreadsLog2 - tx_log2) * col_tiles;
        for (int64_t unit = blockIdx.x; unit < units; unit += sum_blocks) {
            const int64_t piece = row_of<WAVE_ROW>(tx_log2, unit / col_tiles);
            const int64_t vec = ((unit % col_tiles) << tx_log2) + (threadIdx.x & ((1 << tx_log2) - 1));
            if (piece < count && vec < vecs) sum_piece<T, G, NT>(grad_y, ld_grad_y, pc, out, piece, vec);
        }
    } else {
        const int64_t tiles = ((int64_t)pc.groups + kFillRows - 1) / kFillRows;
        for (int64_t t = blockIdx.x - sum_blocks; t < tiles; t += kMaxGridX)
            fill_rows<G>(pc, out, t, fill_tx_log2);
    }
}

// Adds the partial sums of each long run, in order: the one of the piece in which it
// begins and those of the pieces after it.  A workgroup takes a run's 128 columns (32
// lanes of four); eight slices of the workgroup add a contiguous part of the pieces
// each, and their sums are joined in order.
constexpr int kJoinLanes = 32;
constexpr int64_t kMaxJoins = 4096;

template <typename G>
__global__ __launch_bounds__(kThreads) void embedding_join_kernel(Pieces pc, GradOut<G> out, int cols_padded)
{
    const uint32_t *__restrict__ keys = pc.keys;
    const int cols = pc.cols;
    const int64_t count = pc.count(), col_tiles = (cols + 4 * kJoinLanes - 1) / (4 * kJoinLanes);
    constexpr int LANES = kJoinLanes, SLICES = kThreads / LANES;
    __shared__ float s_sum[SLICES][LANES][4];
    __shared__ int64_t s_more;
    const int lane = threadIdx.x & (LANES - 1), slice = threadIdx.x / LANES;
    const int64_t units = (int64_t)pc.list[0] * col_tiles;
    for (int64_t unit = blockIdx.x; unit < units; unit += kMaxJoins) {
        const int64_t piece = pc.list[1 + unit / col_tiles];
        const uint32_t run = keys[(piece + 1) * pc.piece];
        if (threadIdx.x < kWave) {  // how many pieces after it begin with the run
            int64_t more = 2;
            for (;;) {
                const int64_t q = piece + 1 + more + threadIdx.x;
                const uint64_t same = __ballot(q < count && keys[q * pc.piece] == run);
                const int on = same == ~0ull ? kWave : __builtin_ctzll(~same);
                more += on;
                if (on < kWave) break;
            }
            if (threadIdx.x == 0) s_more = more;
        }
        __syncthreads();
        const int64_t c = ((unit % col_tiles) * LANES + lane) * 4;
        // parts 0 .. s_more: the first piece's slot 1, then slot 0 of those after it
        const int64_t parts = s_more + 1, per = (parts + SLICES - 1) / SLICES;
        const int64_t from = slice * per, to = from + per < parts ? from + per : parts;
        float sum[4] = {};
        if (c < cols) {
#pragma unroll 8
            for (int64_t q = from; q < to; ++q) {
                const u32x4 r = *reinterpret_cast<const u32x4 *>(pc.partial +
                                                                       ((piece + q) * 2 + (q == 0)) * cols_padded + c);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += element<float>(r, e);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s_sum[slice][lane][e] = sum[e];
        __syncthreads();
        if (slice == 0 && c < cols) {
            const int64_t used = (parts + per - 1) / per;
            for (int64_t w = 1; w < used; ++w)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += s_sum[w][lane][e];
            // (four columns are half a vector of 16-bit elements: element by element)
            G *p = out.grad + (int64_t)run * out.ld + c;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < cols)
                    p[e] = (G)(out.accumulate ? __builtin_fmaf(out.scale, sum[e], (float)p[e]) : out.scale * sum[e]);
        }
        __syncthreads();
    }
}

}  // namespace lrs_rows
