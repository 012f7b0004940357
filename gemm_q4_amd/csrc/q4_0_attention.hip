// Attention of a ragged batch over the paged cache.
//
// Rows.  A work item is a tile of rows of one conversation and one key/value
// head: row r is query head r % G of that key/value head (G heads share it) and
// new token r / G.  All rows of a tile read the same keys, so a key is read
// once for a group's G heads, for a decode step as for a prefill pass.
//
// Arithmetic (per wave, 32 rows).  Scores are formed transposed, S^T = K Q^T,
// with v_mfma_f32_32x32x16_f16: K from LDS is the A operand, Q stays in
// registers as the B operand, and lane l holds row l % 32's scores of the keys
// 8 a + 4 (l / 32) + 0..3.  The softmax of a row then lives in two lanes: maximum
// and sum are plain register arithmetic and one exchange of wave halves.  The
// weights, rounded to binary16, are as they lie the B operand of
// O^T = V^T P^T, whose A operand (four keys of one column to a lane) the
// transposing LDS read delivers from row-major V.  No value crosses lanes
// between the two products, and O^T's columns are the lane's own row, so the
// running maximum rescales it by a per-lane factor.
//
// Float32 rows split q and the weights into binary16 high and low parts (two
// products each): 22 bits, since K and V are binary16 exactly.
//
// Keys come through LDS by direct copies, in groups of 16 rows (a group never
// crosses a page), the 16-byte pieces of row `key` XOR-swizzled by swz(key) so
// that both kinds of LDS read touch every bank once.  Only groups that some row
// of the tile sees are read; a row of a group that none sees is taken from a
// zero block, so whatever a page holds past its conversation's end never meets
// the arithmetic.
#include "q4_0_device.h"
#include "q4_0_dma.h"
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
// Weights are held as 2^kShift exp(s - m): with m allowed to lag behind the
// true maximum by kLag (in powers of two) before the accumulators are rescaled,
// the largest is 2^15 < 65504, and the smallest binary16 step is 2^-32 of it.
constexpr float kShift = 7.0f, kLag = 8.0f;

// The work of a launch, as the kernels and the joining kernel see it.
struct Plan {
    int group;      // query heads per key/value head
    int splits;     // parts of the key axis
    float *part;    // splits > 1: unnormalised rows [split][n * q_heads][dim]
    float *part_ml; // and their (maximum, sum) [split][n * q_heads][2]
};

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

// A factor applied where the value is a number: an infinity a row earned stays
// one when the factor has vanished.
__device__ __forceinline__ float scaled(float x, float f) {
    return __builtin_isfinite(x) ? x * f : x;
}

// The conversation whose tiles of R rows include tile `w` of the launch, and
// the tile's index within it.  Conversation s is given the tiles from
// q_start[s] G / R + s on: never fewer than its rows need, and known without a
// sum over the conversations before it.
struct Place {
    int s, first, rows, tile;  // first token, rows of the conversation
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
    p.s = find_last(a.batch, [&](int s) {
        return (int64_t)min(max(a.q_start[s], 0), a.n) * group / R + s <= w;
    });
    const meta_t qs = meta(a.q_start);
    p.first = min(max(qs[p.s], 0), a.n);
    const int end = min(max(qs[p.s + 1], p.first), a.n);
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

// Copies of 16 key rows into LDS.  One copy moves 1 KB (512 / DIM rows).
template <int DIM> struct Filler {
    static constexpr int kCopies = DIM / 32;
    static constexpr int kBytes = 16 * DIM * 2;
    uint32_t off[kCopies];
    const AttentionArgs &a;
    const int32_t *table;
    int head;
    __device__ __forceinline__ Filler(const AttentionArgs &args, int s, int hk)
        : a(args), table(args.table + (int64_t)s * args.table_stride), head(hk) {
        const int lane = threadIdx.x % 64;
#pragma unroll
        for (int j = 0; j < kCopies; ++j) {
            const int row = j * (512 / DIM) + lane / (DIM / 8);
            off[j] = row * DIM * 2 + ((lane % (DIM / 8)) ^ swz<DIM>(row)) * 16;
        }
    }
    // Keys k .. k + 15 of K and V; true if every copy was issued.  `parts`: 1 K,
    // 2 V, 3 both.
    template <int KT>
    __device__ __forceinline__ bool fill(const Reach<KT> &r, int k, uint8_t *kbuf, uint8_t *vbuf,
                                         int parts) {
        const int lane = threadIdx.x % 64;
        uint32_t blank = 0;
        if (!r.none(k, 16)) {
            const int shift = a.cache.page_shift;
            const int slot = k >> shift;
            int page = -1;
            if (slot < a.table_stride) page = meta(table)[slot];
            if (page >= 0 && page < a.cache.pages) {
                const int64_t row = (((int64_t)page * a.cache.heads + head) << shift) +
                                    (k & ((1 << shift) - 1));
                const uint8_t *ks = (const uint8_t *)(a.cache.k + row * DIM);
                const uint8_t *vs = (const uint8_t *)(a.cache.v + row * DIM);
                if (r.each(k, 16)) {
                    if (parts & 1)
#pragma unroll
                        for (int j = 0; j < kCopies; ++j) dma16_at(ks, off[j], kbuf + j * 1024);
                    if (parts & 2)
#pragma unroll
                        for (int j = 0; j < kCopies; ++j) dma16_at(vs, off[j], vbuf + j * 1024);
                } else {
#pragma unroll
                    for (int j = 0; j < kCopies; ++j) {
                        const int row16 = j * (512 / DIM) + lane / (DIM / 8);
                        const bool seen = r.any(k + row16);
                        if (parts & 1)
                            dma16(seen ? (const void *)(ks + off[j]) : (const void *)&kZeroPiece,
                                  kbuf + j * 1024);
                        if (parts & 2)
                            dma16(seen ? (const void *)(vs + off[j]) : (const void *)&kZeroPiece,
                                  vbuf + j * 1024);
                    }
                }
                return true;
            }
            blank = 0x7E007E00u;  // no such page: NaN keys for the rows that see them
        }
        const u4_t kv = {blank, blank, blank, blank}, zero = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < kCopies; ++j) {
            if (parts & 1) *(u4_t *)(kbuf + j * 1024 + lane * 16) = kv;
            if (parts & 2) *(u4_t *)(vbuf + j * 1024 + lane * 16) = zero;
        }
        return false;
    }
};

// One wave's 32 rows: its queries, running maximum (of scale log2(e) q.k), sum
// (this lane's half of the keys) and unnormalised result.
template <int DIM, bool F32> struct Rows {
    static constexpr int kParts = F32 ? 2 : 1;
    h8_t q[kParts][DIM / 16];
    f16x_t o[DIM / 32];
    float m, l;
    int p, lo;  // position, first key of the window

    __device__ __forceinline__ void clear() {
        m = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
    }

    // Row r (of the conversation's `rows`); rows past the end repeat the last.
    __device__ __forceinline__ void load(const AttentionArgs &a, const Place &pl, int group,
                                         int hk, int r, int position0) {
        const int half = threadIdx.x % 64 / 32;
        const int rr = min(r, pl.rows - 1);
        const int token = rr / group;
        p = position(a, position0, token);
        lo = a.window && p >= a.window ? p - a.window + 1 : 0;
        const int64_t at = (int64_t)(pl.first + token) * a.q_stride +
                           (int64_t)(hk * group + rr % group) * DIM + 8 * half;
#pragma unroll
        for (int s = 0; s < DIM / 16; ++s) {
            if (!F32) {
                q[0][s] = *(const h8_t *)((const _Float16 *)a.q + at + 16 * s);
            } else {
                const float *x = (const float *)a.q + at + 16 * s;
                const f4_t x0 = *(const f4_t *)x, x1 = *(const f4_t *)(x + 4);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = i < 4 ? x0[i & 3] : x1[i & 3];
                    const _Float16 hi = (_Float16)v;
                    q[0][s][i] = hi;
                    q[kParts - 1][s][i] = (_Float16)(v - (float)hi);
                }
            }
        }
        clear();
    }

    __device__ __forceinline__ bool sees(int key, int sinks) const {
        return key <= p && (key >= lo || key < sinks);
    }

    // KT keys from k0 on, in LDS.  masked: some row sees not all of them.
    // CAREFUL: values that are no numbers touch only the rows that see them.
    template <int KT, bool CAREFUL>
    __device__ __forceinline__ void step(const uint8_t *kbuf, const uint8_t *vbuf, int k0,
                                         bool masked, int sinks, float c) {
        const int lane = threadIdx.x % 64, half = lane / 32;
        f16x_t s[KT / 32];
#pragma unroll
        for (int t = 0; t < KT / 32; ++t) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[t][i] = 0.0f;
            const int key = lane % 32;
            const uint8_t *row = kbuf + (t * 32 + key) * DIM * 2;
#pragma unroll
            for (int d = 0; d < DIM / 16; ++d) {
                const h8_t k = *(const h8_t *)(row + (((2 * d + half) ^ swz<DIM>(key)) * 16));
#pragma unroll
                for (int x = 0; x < kParts; ++x)
                    s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[x][d], s[t], 0, 0, 0);
            }
        }
        if (masked || CAREFUL) {
#pragma unroll
            for (int t = 0; t < KT / 32; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!sees(k0 + t * 32 + 8 * (i / 4) + 4 * half + i % 4, sinks))
                        s[t][i] = -INFINITY;
        }
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < KT / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
        top = halves_max(top) * c;
        if (__any(top > m + kLag)) {
            const float mn = fmaxf(m, top);
            const float f = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] = CAREFUL ? scaled(o[d][i], f) : o[d][i] * f;
        }
        const float base = m == -INFINITY ? 0.0f : kShift - m;
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < KT / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[t][i] = __builtin_amdgcn_exp2f(fmaf(s[t][i], c, base));
                sum += s[t][i];
            }
        l += sum;
#pragma unroll
        for (int b = 0; b < KT / 16; ++b) {
            h8_t w[kParts];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = s[b / 2][8 * (b % 2) + i];
                w[0][i] = (_Float16)x;
                if (F32) w[kParts - 1][i] = (_Float16)(x - (float)w[0][i]);
            }
            const int key = 16 * b + 4 * half + lane % 16 / 4;
            const int piece = 2 * (lane / 16 % 2) + lane % 4 / 2;
            const uint8_t *r0 = vbuf + key * DIM * 2 + 8 * (lane % 2);
            const uint8_t *r1 = r0 + 8 * DIM * 2;
#pragma unroll
            for (int d = 0; d < DIM / 32; ++d) {
                const s4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s4_t)(r0 + ((4 * d + piece) ^ swz<DIM>(key)) * 16));
                const s4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s4_t)(r1 + ((4 * d + piece) ^ swz<DIM>(key + 8)) * 16));
                h8_t v;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = __builtin_bit_cast(_Float16, (short)(i < 4 ? v0[i & 3] : v1[i & 3]));
                if (CAREFUL) {
                    // what is no number leaves the product; rows that see it
                    // are given it afterwards (both signs: NaN)
                    h8_t up, down, see;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float x = (float)v[i];
                        const bool bad = !__builtin_isfinite(x);
                        up[i] = (_Float16)(bad && !(x < 0.0f) ? 1.0f : 0.0f);
                        down[i] = (_Float16)(bad && !(x > 0.0f) ? 1.0f : 0.0f);
                        see[i] = (_Float16)(
                            sees(k0 + 16 * b + 8 * (i / 4) + 4 * half + i % 4, sinks) ? 1.0f
                                                                                      : 0.0f);
                        if (bad) v[i] = (_Float16)0.0f;
                    }
                    f16x_t zero;
#pragma unroll
                    for (int i = 0; i < 16; ++i) zero[i] = 0.0f;
                    const f16x_t u =
                        __builtin_amdgcn_mfma_f32_32x32x16_f16(up, see, zero, 0, 0, 0);
                    const f16x_t w2 =
                        __builtin_amdgcn_mfma_f32_32x32x16_f16(down, see, zero, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (u[i] > 0.0f) o[d][i] += INFINITY;
                        if (w2[i] > 0.0f) o[d][i] -= INFINITY;
                    }
                }
#pragma unroll
                for (int x = 0; x < kParts; ++x)
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, w[x], o[d], 0, 0, 0);
            }
        }
    }

    // Whether a product met something that is no number.
    __device__ __forceinline__ bool odd() const {
        float z = l * 0.0f;
#pragma unroll
        for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) z += o[d][i] * 0.0f;
        return !(z == 0.0f);
    }
};

// The rows' results, to y or to this split's share of the workspace.  `o` holds
// four neighbouring elements of row `row` from element d on.
template <bool F32>
__device__ __forceinline__ void put4(const AttentionArgs &a, const Plan &pl, int split,
                                     int64_t row, int dim, int d, f4_t o, float l, bool sees) {
    if (pl.splits > 1) {
        *(f4_t *)(pl.part + ((int64_t)split * a.n * a.q_heads + row) * dim + d) = o;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = sees ? o[i] / l : 0.0f;
    if (F32)
        *(f4_t *)((float *)a.y + row * dim + d) = o;
    else
        *(h4_t *)((_Float16 *)a.y + row * dim + d) =
            h4_t{(_Float16)o[0], (_Float16)o[1], (_Float16)o[2], (_Float16)o[3]};
}

__device__ __forceinline__ void put_ml(const AttentionArgs &a, const Plan &pl, int split,
                                       int64_t row, float m, float l) {
    float *ml = pl.part_ml + ((int64_t)split * a.n * a.q_heads + row) * 2;
    ml[0] = m;
    ml[1] = l;
}

// ---- many rows: four waves of 32 rows share each key tile -------------------
// Two stages of KT keys in LDS: while the waves work on one, the copies of the
// next are in flight.
template <int DIM> constexpr int kPassKeys = DIM > 128 ? 32 : 64;
constexpr int kPassRows = 128;

template <int DIM, bool F32, bool CAREFUL>
__device__ __forceinline__ void pass_loop(Rows<DIM, F32> &w, Filler<DIM> &f,
                                          const Reach<kPassKeys<DIM>> &r, int t0, int t1,
                                          int top_lo, float c, uint8_t *lds) {
    constexpr int KT = kPassKeys<DIM>;
    constexpr int kTile = KT * DIM * 2;
    const int wave = uniform(threadIdx.x / 64);
    const auto fill = [&](int t, int stage) {
        uint8_t *kbuf = lds + stage * 2 * kTile, *vbuf = kbuf + kTile;
        const int k = r.key(t);
        if (KT == 64) {
            const int at = 16 * wave;
            f.fill(r, k + at, kbuf + at * DIM * 2, vbuf + at * DIM * 2, 3);
        } else {
            const int at = 16 * (wave % 2);
            f.fill(r, k + at, kbuf + at * DIM * 2, vbuf + at * DIM * 2, wave < 2 ? 1 : 2);
        }
    };
    fill(t0, 0);
    for (int t = t0; t < t1; ++t) {
        const int stage = (t - t0) & 1;
        Q4_WAIT_VMCNT(0);
        __syncthreads();
        if (t + 1 < t1) fill(t + 1, stage ^ 1);
        const int k = r.key(t);
        const uint8_t *kbuf = lds + stage * 2 * kTile;
        w.template step<KT, CAREFUL>(kbuf, kbuf + kTile, k, !r.all(k, KT, top_lo), r.sinks, c);
    }
}

template <int DIM, bool F32>
__global__ __launch_bounds__(256, DIM > 128 ? 1 : 2) void pass_kernel(AttentionArgs a, Plan pl, int base) {
    constexpr int KT = kPassKeys<DIM>;
    __shared__ __align__(1024) uint8_t lds[2 * 2 * KT * DIM * 2];
    const int hk = blockIdx.x % a.cache.heads;
    const int rest = blockIdx.x / a.cache.heads;
    const int split = rest % pl.splits;
    Place at = find_tile<kPassRows>(a, pl.group, base + rest / pl.splits);
    const int count = (at.rows + kPassRows - 1) / kPassRows;
    if (at.tile < 0 || at.tile >= count) return;
    at.tile = count - 1 - at.tile;  // the tiles with the most keys first
    const int kv = max(meta(a.kv_len)[at.s], 0);
    const int position0 = kv - at.rows / pl.group;
    const int row0 = at.tile * kPassRows, row1 = min(row0 + kPassRows, at.rows);
    const int p0 = position(a, position0, row0 / pl.group);
    const int p1 = position(a, position0, (row1 - 1) / pl.group);
    const Reach<KT> r(a, p0, p1);
    const int top_lo = a.window && p1 >= a.window ? p1 - a.window + 1 : 0;
    const int per = (r.tiles + pl.splits - 1) / pl.splits;
    const int t0 = min(split * per, r.tiles), t1 = min(t0 + per, r.tiles);
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int row = row0 + wave * 32 + lane % 32;
    Rows<DIM, F32> w;
    w.load(a, at, pl.group, hk, row, position0);
    if (t0 < t1) {
        Filler<DIM> f(a, at.s, hk);
        const float c = a.scale * kLog2e;
        pass_loop<DIM, F32, false>(w, f, r, t0, t1, top_lo, c, lds);
        if (__syncthreads_or(w.odd())) {
            w.clear();
            pass_loop<DIM, F32, true>(w, f, r, t0, t1, top_lo, c, lds);
        }
    }
    if (row >= row1) return;
    const float l = halves_sum(w.l);
    const int64_t out = (int64_t)(at.first + row / pl.group) * a.q_heads + hk * pl.group +
                        row % pl.group;
    const int half = lane / 32;
    if (pl.splits > 1) {
        if (half == 0) put_ml(a, pl, split, out, w.m, l);
        if (t0 >= t1) return;
    }
#pragma unroll
    for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            put4<F32>(a, pl, split, out, DIM, 32 * d + 2 * i + 4 * half,
                      f4_t{w.o[d][i], w.o[d][i + 1], w.o[d][i + 2], w.o[d][i + 3]}, l,
                      w.p >= 0);
}

// ---- few rows: every wave streams its own keys for the same 32 rows ---------
// No barrier in the loop: a wave fills its own two stages and waits for its own
// copies.  The waves' results are joined through LDS at the end.
constexpr int kStepRows = 32, kStepKeys = 32;
template <int DIM> constexpr int kStepWaves = DIM > 128 ? 2 : 4;

template <int DIM, bool F32, bool CAREFUL>
__device__ __forceinline__ void step_loop(Rows<DIM, F32> &w, Filler<DIM> &f,
                                          const Reach<kStepKeys> &r, int t0, int t1, int stride,
                                          int top_lo, float c, uint8_t *lds) {
    constexpr int KT = kStepKeys;
    constexpr int kTile = KT * DIM * 2;
    constexpr int kCopies = KT / 16 * 2 * Filler<DIM>::kCopies;
    const auto fill = [&](int t, int stage) {
        uint8_t *kbuf = lds + stage * 2 * kTile, *vbuf = kbuf + kTile;
        const int k = r.key(t);
        bool full = true;
#pragma unroll
        for (int at = 0; at < KT; at += 16)
            full &= f.fill(r, k + at, kbuf + at * DIM * 2, vbuf + at * DIM * 2, 3);
        return full;
    };
    if (t0 >= t1) return;
    fill(t0, 0);
    int stage = 0;
    for (int t = t0; t < t1; t += stride) {
        bool counted = false;
        if (t + stride < t1) counted = fill(t + stride, stage ^ 1);
        if (counted)
            Q4_WAIT_VMCNT(kCopies);
        else
            Q4_WAIT_VMCNT(0);
        asm volatile("" ::: "memory");
        const int k = r.key(t);
        const uint8_t *kbuf = lds + stage * 2 * kTile;
        w.template step<KT, CAREFUL>(kbuf, kbuf + kTile, k, !r.all(k, KT, top_lo), r.sinks, c);
        Q4_WAIT_LGKM0();
        asm volatile("" ::: "memory");
        stage ^= 1;
    }
}

template <int DIM, bool F32>
__global__ __launch_bounds__(64 * kStepWaves<DIM>) void step_kernel(AttentionArgs a, Plan pl, int base) {
    constexpr int KT = kStepKeys, W = kStepWaves<DIM>;
    constexpr int kStage = 2 * KT * DIM * 2;  // K and V
    constexpr int kPitch = DIM + 4;
    __shared__ __align__(1024) uint8_t lds[W * 2 * kStage];
    __shared__ float ml[2][W][32];
    static_assert(32 * kPitch * 4 <= 2 * kStage, "a wave's rows fit its own stages");
    const int hk = blockIdx.x % a.cache.heads;
    const int rest = blockIdx.x / a.cache.heads;
    const int split = rest % pl.splits;
    const Place at = find_tile<kStepRows>(a, pl.group, base + rest / pl.splits);
    const int row0 = at.tile * kStepRows;
    if (row0 < 0 || row0 >= at.rows) return;
    const int row1 = min(row0 + kStepRows, at.rows);
    const int kv = max(meta(a.kv_len)[at.s], 0);
    const int position0 = kv - at.rows / pl.group;
    const int p0 = position(a, position0, row0 / pl.group);
    const int p1 = position(a, position0, (row1 - 1) / pl.group);
    const Reach<KT> r(a, p0, p1);
    const int top_lo = a.window && p1 >= a.window ? p1 - a.window + 1 : 0;
    const int per = (r.tiles + pl.splits - 1) / pl.splits;
    const int t0 = min(split * per, r.tiles), t1 = min(t0 + per, r.tiles);
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    Rows<DIM, F32> w;
    w.load(a, at, pl.group, hk, row0 + lane % 32, position0);
    uint8_t *mine = lds + wave * 2 * kStage;
    Filler<DIM> f(a, at.s, hk);
    const float c = a.scale * kLog2e;
    step_loop<DIM, F32, false>(w, f, r, t0 + wave, t1, W, top_lo, c, mine);
    if (__any(w.odd())) {
        w.clear();
        step_loop<DIM, F32, true>(w, f, r, t0 + wave, t1, W, top_lo, c, mine);
    }
    // join the waves
    w.l = halves_sum(w.l);
    if (lane < 32) ml[0][wave][lane] = w.m, ml[1][wave][lane] = w.l;
    __syncthreads();
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) m = fmaxf(m, ml[0][i][lane % 32]);
    const float fs = w.m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(w.m - m);
    float *rows = (float *)mine;
#pragma unroll
    for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            f4_t v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = scaled(w.o[d][i + e], fs);
            *(f4_t *)(rows + (lane % 32) * kPitch + 32 * d + 2 * i + 4 * (lane / 32)) = v;
        }
    __syncthreads();
    for (int e = threadIdx.x; e < (row1 - row0) * (DIM / 4); e += 64 * W) {
        const int rr = e / (DIM / 4), d = e % (DIM / 4) * 4;
        f4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
        m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) m = fmaxf(m, ml[0][i][rr]);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const f4_t v = *(const f4_t *)((const float *)(lds + i * 2 * kStage) + rr * kPitch + d);
#pragma unroll
            for (int x = 0; x < 4; ++x) o[x] += v[x];
            if (ml[0][i][rr] != -INFINITY || ml[1][i][rr] != 0.0f)
                l += scaled(ml[1][i][rr], __builtin_amdgcn_exp2f(ml[0][i][rr] - m));
        }
        const int token = (row0 + rr) / pl.group;
        const int64_t out = (int64_t)(at.first + token) * a.q_heads + hk * pl.group +
                            (row0 + rr) % pl.group;
        if (pl.splits > 1 && d == 0) put_ml(a, pl, split, out, m, l);
        if (pl.splits > 1 && t0 >= t1) continue;
        put4<F32>(a, pl, split, out, DIM, d, o, l, position0 + token >= 0);
    }
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
    const int64_t row = blockIdx.x;
    const int token = (int)(row / a.q_heads), dim = a.cache.dim;
    // the last conversation that starts at or before the token
    const int s = find_last(a.batch, [&](int i) { return a.q_start[i] <= token; });
    const meta_t qs = meta(a.q_start);
    const int first = min(max(qs[s], 0), a.n), end = min(max(qs[s + 1], first), a.n);
    if (token < first || token >= end) return;
    const bool sees = max(meta(a.kv_len)[s], 0) - end + token >= 0;
    const int x = threadIdx.x, wave = x / 64;
    float m = -INFINITY, l = 0.0f;
    if (x < pl.splits) {
        const float *ml = pl.part_ml + ((int64_t)x * a.n * a.q_heads + row) * 2;
        m = ml[0], l = ml[1];
    }
    float top = m;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) top = fmaxf(top, __shfl_xor(top, i));
    if (x % 64 == 0) wave_m[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(wave_m[0], wave_m[1]), fmaxf(wave_m[2], wave_m[3]));
    // a part that saw none of the row's keys wrote no elements: marked by -1
    const bool used = m != -INFINITY || l != 0.0f;
    const float f = used ? __builtin_amdgcn_exp2f(m - top) : -1.0f;
    if (x < pl.splits) factor[x] = f;
    l = used ? scaled(l, f) : 0.0f;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) l += __shfl_xor(l, i);
    if (x % 64 == 0) wave_l[wave] = l;
    __syncthreads();
    l = wave_l[0] + wave_l[1] + wave_l[2] + wave_l[3];
    const int cols = dim / 4, col = x % cols;
    f4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = x / cols; i < pl.splits; i += 256 / cols) {
        const float g = factor[i];
        if (g == -1.0f) continue;
        const f4_t v =
            *(const f4_t *)(pl.part + ((int64_t)i * a.n * a.q_heads + row) * dim + col * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += scaled(v[e], g);
    }
    sums[x] = o;
    __syncthreads();
    if (x >= cols) return;
    for (int i = x + cols; i < 256; i += cols) {
        const f4_t v = sums[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += v[e];
    }
    Plan whole = pl;
    whole.splits = 1;
    put4<F32>(a, whole, 0, row, dim, 4 * x, o, l, sees);
}

// ---- choices on the host ----------------------------------------------------
struct Choice {
    bool pass;  // 128-row tiles; else 32-row ones, every wave on its own keys
    int64_t tiles;
    int splits;
    size_t part, bytes;  // workspace: bytes of the partial rows, and in all
};

Choice choose(const AttentionArgs &a) {
    Choice ch;
    const int dim = a.cache.dim, heads = a.cache.heads;
    const int64_t rows = (int64_t)a.n * (a.q_heads / heads);
    // more rows to a conversation than a 32-row tile holds: the waves share
    // the keys; up to that they share the rows and split the keys
    ch.pass = rows > (int64_t)kStepRows * a.batch;
    const int R = ch.pass ? kPassRows : kStepRows;
    ch.tiles = rows / R + a.batch;
    const int64_t likely = (ch.pass ? rows / R + (a.batch + 1) / 2
                                    : (rows / R > a.batch ? rows / R : a.batch)) *
                           heads;
    // the key tiles a row tile can have at most
    const int KT = ch.pass ? (dim > 128 ? kPassKeys<256> : kPassKeys<128>) : kStepKeys;
    int64_t keys = (int64_t)a.table_stride << a.cache.page_shift;
    if (a.window) {
        const int64_t near = (int64_t)a.window + a.sinks + 2 * R + 2 * KT;
        if (near < keys) keys = near;
    }
    const int64_t most = (keys + KT - 1) / KT;
    const int waves = dim > 128 ? kStepWaves<256> : kStepWaves<128>;
    const int64_t slots = (int64_t)device_shape().cus * (ch.pass ? (dim > 128 ? 1 : 2)
                                                                 : (dim > 64 ? 1 : 2));
    int64_t splits = likely >= slots ? 1 : slots / likely;
    const int64_t least = ch.pass ? 4 : 2 * waves;  // tiles a part should have
    if (splits > most / least) splits = most / least;
    if (splits > kMaxSplits) splits = kMaxSplits;
    const int64_t out = (int64_t)a.n * a.q_heads;
    const int64_t room = (int64_t)kWorkspaceBytes / (out * (dim + 2) * 4);
    if (splits > room) splits = room;
    ch.splits = splits < 2 ? 1 : (int)splits;
    ch.part = ch.splits > 1 ? (size_t)ch.splits * (size_t)out * (size_t)dim * 4u : 0;
    ch.bytes = ch.splits > 1 ? ch.part + (size_t)ch.splits * (size_t)out * 8u : 0;
    return ch;
}

template <int DIM, bool F32>
hipError_t run(const AttentionArgs &a, const Choice &ch, const Plan &pl, hipStream_t stream) {
    // a launch's work items stay below 2^31
    const int64_t each = (INT64_C(1) << 22) / (ch.splits * a.cache.heads);
    for (int64_t base = 0; base < ch.tiles; base += each) {
        const int64_t tiles = ch.tiles - base < each ? ch.tiles - base : each;
        const dim3 grid((uint32_t)(tiles * ch.splits * a.cache.heads));
        if (ch.pass)
            hipLaunchKernelGGL((pass_kernel<DIM, F32>), grid, dim3(256), 0, stream, a, pl,
                               (int)base);
        else
            hipLaunchKernelGGL((step_kernel<DIM, F32>), grid, dim3(64 * kStepWaves<DIM>), 0,
                               stream, a, pl, (int)base);
    }
    if (ch.splits > 1)
        hipLaunchKernelGGL((join_kernel<F32>), dim3((uint32_t)(a.n * a.q_heads)), dim3(256), 0,
                           stream, a, pl);
    return hipGetLastError();
}

template <bool F32>
hipError_t by_dim(const AttentionArgs &a, const Choice &ch, const Plan &pl, hipStream_t stream) {
    if (a.cache.dim == 64) return run<64, F32>(a, ch, pl, stream);
    if (a.cache.dim == 128) return run<128, F32>(a, ch, pl, stream);
    return run<256, F32>(a, ch, pl, stream);
}

}  // namespace

bool attention_supports(int dim) { return dim == 64 || dim == 128 || dim == 256; }

size_t attention_workspace_bytes(const AttentionArgs &a, int) { return choose(a).bytes; }

hipError_t launch_attention(const AttentionArgs &a, int x_f16, void *ws, hipStream_t stream) {
    const Choice ch = choose(a);
    const Plan pl = {a.q_heads / a.cache.heads, ch.splits, (float *)ws,
                     (float *)((uint8_t *)ws + ch.part)};
    return x_f16 ? by_dim<false>(a, ch, pl, stream) : by_dim<true>(a, ch, pl, stream);
}

}  // namespace q4
