// What the attention kernels over binary16 and over 8-bit caches share: finding a
// tile's rows and keys in a ragged batch, the rows' results, and joining the
// parts of a split key axis.
#pragma once

#include <float.h>

#include "q4_0_device.h"
#include "q4_0_internal.h"

namespace q4 {

namespace {

typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
typedef short s4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4_t *lds_s4_t;
// the metadata is read by scalar loads: they do not mix with the count of the
// direct copies in flight
typedef const __attribute__((address_space(4))) int32_t *meta_t;

constexpr float kLog2e = 1.4426950408889634f;
// The work of a launch, as the kernels and the joining kernel see it.
struct Plan {
    int group;      // query heads per key/value head
    int splits;     // parts of the key axis, at most
    int least;      // key tiles of a part, at least
    float *part;    // splits > 1: unnormalised rows [split][n * q_heads][dim]
    float *part_ml; // and their (maximum, sum) [split][n * q_heads][2]
};

// Where 16-byte piece p of binary16 key row `key` lies in an LDS tile: p ^ swz(key).
template <int DIM> __device__ __forceinline__ int swz(int key) {
    // 256-byte spans of LDS hold one row (two at 64 elements): 16 keys at one
    // piece, and 4 keys at 4 neighbouring pieces, both fall on distinct banks
    if (DIM >= 128) return ((key & 3) << 2) | ((key >> 2) & 3);
    return (((key >> 1) & 1) << 2) | ((key >> 2) & 3);
}

__device__ __forceinline__ meta_t meta(const int32_t *p) { return (meta_t)(uintptr_t)p; }

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// x of the other half of the wave joined by max or sum.
__device__ __forceinline__ float halves_max(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]),
                 __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float halves_sum(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// exp2 of a difference of maxima, never 0: an infinity that a row earned
// stays one, and what a vanished factor scales is far below a float32 step of
// the sum it joins.
__device__ __forceinline__ float factor_of(float d) {
    return fmaxf(__builtin_amdgcn_exp2f(d), 2e-38f);
}

// The factor of scores, kept a number other than 0 whatever scale and q are: as 0
// it would make a masked score (minus infinity) NaN, as infinity a score of 0.
// Below this range every visible key weighs the same, above it only equal
// scores do, with the factor or without.
__device__ __forceinline__ float finite(float c) {
    return __builtin_amdgcn_fmed3f(c, FLT_MIN, FLT_MAX);
}

// The conversation whose tiles of R rows include tile `w` of the launch, and
// the tile's index within it.  Conversation s is given the tiles from
// q_start[s] G / R + s on: never fewer than its rows need, and known without a
// sum over the conversations before it.
struct Place {
    int s, first, rows, tile;  // first token and rows of the conversation
    int kv;                    // its length
};

// The last i < count with holds(i), where holds is true up to some index and
// false from there on (0 if it is never true).  64 lanes look at once.
template <typename F> __device__ __forceinline__ int find_last(int count, F holds) {
    const int lane = threadIdx.x % 64;
    int lo = 0, hi = count;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64;
        const int i = lo + lane * step;
        const int last = __popcll(__ballot(i < hi && holds(i))) - 1;
        lo += (last < 0 ? 0 : last) * step;
        hi = min(lo + step, hi);
    }
    return uniform(lo);
}

template <int R>
__device__ __forceinline__ Place find_tile(const AttentionArgs &a, int group, int w) {
    Place p;
    int end;
    if (a.batch <= 64) {
        // every lane's conversation in one round of loads
        const int s = min((int)(threadIdx.x % 64), a.batch - 1);
        const int b = min(max(a.q_start[s], 0), a.n), e = a.q_start[s + 1], kv = a.kv_len[s];
        const bool below = (int64_t)b * group / R + s <= w && (int)(threadIdx.x % 64) < a.batch;
        const int last = __popcll(__ballot(below)) - 1;
        p.s = uniform(last < 0 ? 0 : last);
        p.first = __builtin_amdgcn_readlane(b, p.s);
        end = __builtin_amdgcn_readlane(e, p.s);
        p.kv = __builtin_amdgcn_readlane(kv, p.s);
    } else {
        p.s = find_last(a.batch, [&](int s) {
            return (int64_t)min(max(a.q_start[s], 0), a.n) * group / R + s <= w;
        });
        const meta_t qs = meta(a.q_start);
        p.first = min(max(qs[p.s], 0), a.n);
        end = qs[p.s + 1];
        p.kv = meta(a.kv_len)[p.s];
    }
    end = min(max(end, p.first), a.n);
    p.kv = max(p.kv, 0);
    p.rows = (end - p.first) * group;
    p.tile = w - (int)((int64_t)p.first * group / R + p.s);
    return p;
}

// Position of a conversation's new token i (negative: it sees nothing).  One
// that lies past the page table sees a key without a page whatever its window
// is; it is taken as the first such position, so that no length, however
// wrong, makes a loop longer than the table.
__device__ __forceinline__ int position(const AttentionArgs &a, int position0, int i) {
    return min(position0 + i, a.table_stride << a.cache.page_shift);
}

// What a tile's rows see: positions of its first and last token, the first key
// of the first token's window, and the key tiles that leaves.
template <int KT> struct Reach {
    int pmin, pmax, lo, sinks;
    int sink_tiles, first_tile, tiles;
    __device__ __forceinline__ Reach(const AttentionArgs &a, int p0, int p1) {
        pmin = p0, pmax = p1, sinks = a.sinks;
        lo = a.window && p0 >= a.window ? p0 - a.window + 1 : 0;
        tiles = sink_tiles = first_tile = 0;
        if (p1 < 0) return;
        const int end = p1 / KT + 1;
        sink_tiles = lo > 0 ? min((int)(((int64_t)sinks + KT - 1) / KT), end) : 0;
        first_tile = max(lo / KT, sink_tiles);
        tiles = sink_tiles + max(end - first_tile, 0);
    }
    __device__ __forceinline__ int key(int t) const {
        return (t < sink_tiles ? t : first_tile + t - sink_tiles) * KT;
    }
    // keys [k, k + count): seen by every row, by none
    __device__ __forceinline__ bool all(int k, int count, int top_lo) const {
        return k + count - 1 <= pmin && (k >= top_lo || k + count <= sinks);
    }
    __device__ __forceinline__ bool any(int k) const {
        return k <= pmax && (k >= lo || k < sinks);
    }
    __device__ __forceinline__ bool none(int k, int count) const {
        return k > pmax || (k + count - 1 < lo && k >= sinks);
    }
    __device__ __forceinline__ bool each(int k, int count) const {
        return k + count - 1 <= pmax && (k >= lo || k + count <= sinks);
    }
};

// The rows' results, to y or to this split's share of the workspace.  `o` holds
// four neighbouring elements of row `row` from element d on.
template <bool F32>
__device__ __forceinline__ void put_y4(const AttentionArgs &a, int64_t row, int dim, int d, f4_t o,
                                       float l, bool sees) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = sees ? o[i] / l : 0.0f;
    if (F32)
        *(f4_t *)((float *)a.y + row * dim + d) = o;
    else
        *(h4_t *)((_Float16 *)a.y + row * dim + d) =
            h4_t{(_Float16)o[0], (_Float16)o[1], (_Float16)o[2], (_Float16)o[3]};
}

template <bool F32>
__device__ __forceinline__ void put4(const AttentionArgs &a, const Plan &pl, int split,
                                     int64_t row, int dim, int d, f4_t o, float l, bool sees) {
    if (pl.splits > 1)
        *(f4_t *)(pl.part + ((int64_t)split * a.n * a.q_heads + row) * dim + d) = o;
    else
        put_y4<F32>(a, row, dim, d, o, l, sees);
}

__device__ __forceinline__ void put_ml(const AttentionArgs &a, const Plan &pl, int split,
                                       int64_t row, float m, float l) {
    float *ml = pl.part_ml + ((int64_t)split * a.n * a.q_heads + row) * 2;
    ml[0] = m;
    ml[1] = l;
}

// ---- joining the parts of the key axis --------------------------------------
// One workgroup per row (token and query head): factors from the parts' maxima,
// then the weighted sum, the parts dealt to the lanes that one column of four
// elements leaves free.
constexpr int kMaxSplits = 256;

template <bool F32>
__global__ __launch_bounds__(256) void join_kernel(AttentionArgs a, Plan pl) {
    __shared__ float factor[kMaxSplits];
    __shared__ float wave_m[4], wave_l[4];
    __shared__ f4_t sums[256];
    const int64_t row = blockIdx.x, rows = (int64_t)a.n * a.q_heads;
    const int token = (int)(row / a.q_heads), dim = a.cache.dim;
    const int x = threadIdx.x, wave = x / 64;
    const int cols = dim / 4, lanes = 256 / cols, first = x / cols;
    // what does not depend on the conversation is requested before it is known;
    // a part that was not written is never used
    constexpr int kAhead = 4;
    f4_t ahead[kAhead];
    const float *src = pl.part + row * dim + x % cols * 4;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int part = first + i * lanes;
        if (part < pl.splits) ahead[i] = *(const f4_t *)(src + part * rows * dim);
    }
    float m = -INFINITY, l = 0.0f;
    if (x < pl.splits) {
        const float *ml = pl.part_ml + (x * rows + row) * 2;
        m = ml[0], l = ml[1];
    }
    // the last conversation that starts at or before the token
    const int s = find_last(a.batch, [&](int i) { return a.q_start[i] <= token; });
    const meta_t qs = meta(a.q_start);
    const int begin = min(max(qs[s], 0), a.n), end = min(max(qs[s + 1], begin), a.n);
    if (token < begin || token >= end) return;
    const bool sees = max(meta(a.kv_len)[s], 0) - end + token >= 0;
    float top = m;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) top = fmaxf(top, __shfl_xor(top, i));
    if (x % 64 == 0) wave_m[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(wave_m[0], wave_m[1]), fmaxf(wave_m[2], wave_m[3]));
    // a part that saw none of the row's keys wrote no elements: marked by -1
    const bool used = m != -INFINITY || l != 0.0f;
    const float f = used ? factor_of(m - (top == -INFINITY ? 0.0f : top)) : -1.0f;
    if (x < pl.splits) factor[x] = f;
    l = used ? l * f : 0.0f;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) l += __shfl_xor(l, i);
    if (x % 64 == 0) wave_l[wave] = l;
    __syncthreads();
    l = wave_l[0] + wave_l[1] + wave_l[2] + wave_l[3];
    f4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
    const auto add = [&](const f4_t &v, int part) {
        const float g = factor[part];
        if (g == -1.0f) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += v[e] * g;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (first + i * lanes < pl.splits) add(ahead[i], first + i * lanes);
    for (int part = first + kAhead * lanes; part < pl.splits; part += lanes)
        add(*(const f4_t *)(src + part * rows * dim), part);
    sums[x] = o;
    __syncthreads();
    if (x >= cols) return;
    for (int i = x + cols; i < 256; i += cols) {
        const f4_t v = sums[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += v[e];
    }
    put_y4<F32>(a, row, dim, 4 * x, o, l, sees);
}

}  // namespace

}  // namespace q4
