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
// products each): 22 bits, since K and V are binary16 exactly.  Few rows (32-row
// tiles) split the weights of binary16 rows too: bound by the bytes, they pay
// nothing for it (64 conversations 182 us either way; 131071 keys 83.5 and 82.5),
// and their results are off by the result's own rounding alone.  Passes round
// such weights once (2^-11): in two parts two prompts took 431 instead of 318 us,
// 512 tokens under a window 23.5 instead of 20.6.
//
// Keys come through LDS by direct copies, in groups of 16 rows (a group never
// crosses a page), the 16-byte pieces of row `key` XOR-swizzled by swz(key) so
// that both kinds of LDS read touch every bank once.  Only groups that some row
// of the tile sees are read; a row of a group that none sees is taken from a
// zero block, so whatever a page holds past its conversation's end never meets
// the arithmetic.
#include "q4_0_attention.h"
#include "q4_0_dma.h"

namespace q4 {

namespace {

// Copies of 16 key rows into LDS.  One copy moves 1 KB (512 / DIM rows).  Pages
// are looked up 64 tiles at a time, one to a lane, so that the loop reads its
// page from a register and never waits for the table.
// ONCE: every key is read by one workgroup, and the copies carry the
// non-temporal hint (131071 keys: 94 us without, 83 us with; 64 conversations
// 206 and 183 us).  Where other tiles read the same keys it gains nothing.
template <int DIM, bool ONCE> struct Filler {
    static constexpr int kCopies = DIM / 32;
    uint32_t off[kCopies];
    const uint8_t *k, *v;  // of this head, on page 0
    const int32_t *table;
    int64_t page_bytes;
    int pages, table_stride, shift;
    __device__ __forceinline__ Filler(const AttentionArgs &a, int s, int hk)
        : table(a.table + (int64_t)s * a.table_stride),
          page_bytes(((int64_t)a.cache.heads << a.cache.page_shift) * DIM * 2),
          pages((int)a.cache.pages), table_stride(a.table_stride), shift(a.cache.page_shift) {
        const int64_t at = ((int64_t)hk << shift) * DIM * 2;
        k = (const uint8_t *)a.cache.k + at;
        v = (const uint8_t *)a.cache.v + at;
#pragma unroll
        for (int j = 0; j < kCopies; ++j) off[j] = offset(j);
    }
    // Byte offset of this lane's piece of copy j within the 16 rows.
    static __device__ __forceinline__ uint32_t offset(int j) {
        const int lane = threadIdx.x % 64;
        const int row = j * (512 / DIM) + lane / (DIM / 8);
        return row * DIM * 2 + ((lane % (DIM / 8)) ^ swz<DIM>(row)) * 16;
    }
    // The page of key `key` (of the lane's own choice), -1 if it has none.
    __device__ __forceinline__ int look(int key) const {
        const int slot = key >> shift;
        const int page = slot < table_stride ? table[slot] : -1;
        return page < pages ? max(page, -1) : -1;
    }
    // Keys key .. key + 15, of K or of V, from page `page` (wave-uniform); true
    // if all its copies were issued and nothing else.
    template <int KT>
    __device__ __forceinline__ bool fill(const Reach<KT> &r, int page, int key, uint8_t *dst,
                                         bool is_v) const {
        const uint8_t *src = (is_v ? v : k) + page * page_bytes +
                             (int64_t)((key & ((1 << shift) - 1)) * (DIM * 2));
        if (__builtin_expect(page >= 0 && r.each(key, 16), 1)) {
#pragma unroll
            for (int j = 0; j < kCopies; ++j) {
                if (ONCE)
                    dma16_once_at(src, off[j], dst + j * 1024);
                else
                    dma16_at(src, off[j], dst + j * 1024);
            }
            return true;
        }
        // No page: NaN keys for the rows that see them.  Rows that no row of
        // the tile sees: zeros.
        const int lane = threadIdx.x % 64;
        const bool unseen = r.none(key, 16);
        const uint32_t x = unseen || is_v ? 0u : 0x7E007E00u;
        const u4_t blank = {x, x, x, x};
#pragma nounroll
        for (int j = 0; j < kCopies; ++j) {
            if (page < 0 || unseen)
                *(u4_t *)(dst + j * 1024 + lane * 16) = blank;
            else
                dma16(r.any(key + j * (512 / DIM) + lane / (DIM / 8))
                          ? (const void *)(src + offset(j))
                          : (const void *)&kZeroPiece,
                      dst + j * 1024);
        }
        return false;
    }
};

// One wave's 32 rows: its queries, running maximum (of scale log2(e) q.k), sum
// (this lane's half of the keys) and unnormalised result.  FINE: weights in two
// parts.
template <int DIM, bool F32, bool FINE> struct Rows {
    static constexpr int kParts = F32 ? 2 : 1;       // of q
    static constexpr int kWeights = FINE ? 2 : 1;    // of a weight
    // Weights are held as 2^kShift exp(s - m), where m may lag behind the true
    // maximum by kLag (in powers of two) before the accumulators are rescaled:
    // 2^15 < 65504 at most.  Binary16's smallest step is then 2^-32 of the
    // largest weight; weights in two parts rescale more often and keep 2^-39, so
    // that a hundred thousand faint ones beside a strong one keep their sum.
    static constexpr float kShift = FINE ? 14.0f : 7.0f, kLag = FINE ? 1.0f : 8.0f;
    static constexpr float kFar = 65536.0f;
    h8_t q[kParts][DIM / 16];
    f16x_t o[DIM / 32];
    float m, l;
    float c;    // scores to powers of two
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
    // take() forms the operands, so that other requests can go out in between.
    struct Raw {
        u4_t x[kParts * DIM / 16];
    };
    __device__ __forceinline__ void request(Raw &raw, const AttentionArgs &a, const Place &pl,
                                            int group, int hk, int r, int position0) {
        const int half = threadIdx.x % 64 / 32;
        const int rr = min(r, pl.rows - 1);
        const int token = rr / group;
        p = position(a, position0, token);
        lo = a.window && p >= a.window ? p - a.window + 1 : 0;
        c = finite(a.scale * kLog2e);
        const int64_t at = (int64_t)(pl.first + token) * a.q_stride +
                           (int64_t)(hk * group + rr % group) * DIM + 8 * half;
        const u4_t *src = (const u4_t *)((const uint8_t *)a.q + at * (F32 ? 4 : 2));
#pragma unroll
        for (int s = 0; s < DIM / 16; ++s)
#pragma unroll
            for (int x = 0; x < kParts; ++x) raw.x[s * kParts + x] = src[s * (F32 ? 4 : 2) + x];
        clear();
    }
    __device__ __forceinline__ void take(const Raw &raw) {
        int e = 0;
        if (F32) {
            // the row's largest element brought into [1/2, 1), so that its parts
            // are neither infinite nor faint whatever q's magnitude
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < kParts * DIM / 4; ++i) {
                const uint32_t bits = raw.x[i / 4][i % 4];
                top = fmaxf(top, fabsf(__builtin_bit_cast(float, bits)));
            }
            e = __builtin_amdgcn_frexp_expf(halves_max(top));
            c = finite(__builtin_amdgcn_ldexpf(c, e));
        }
#pragma unroll
        for (int s = 0; s < DIM / 16; ++s) {
            if (!F32) {
                q[0][s] = __builtin_bit_cast(h8_t, raw.x[s]);
                continue;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // (a bit cast of the vector's element itself reads element 0)
                const uint32_t bits = raw.x[s * kParts + (i / 4) % kParts][i % 4];
                const float v = __builtin_amdgcn_ldexpf(__builtin_bit_cast(float, bits), -e);
                const _Float16 hi = (_Float16)v;
                q[0][s][i] = hi;
                q[kParts - 1][s][i] = (_Float16)(v - (float)hi);
            }
        }
    }

    __device__ __forceinline__ bool sees(int key, int sinks) const {
        return key <= p && (key >= lo || key < sinks);
    }

    // Scores of KT keys from k0 on, K in LDS.  masked: some row sees not all of
    // them.  CAREFUL: bit i of `gone` is set where score i is minus infinity.
    // The high parts of float32 queries alone decide that: beside an infinite
    // key the low parts, 0 or of either sign, make NaN.
    template <int KT, bool CAREFUL>
    __device__ __forceinline__ uint32_t scores(f16x_t (&s)[KT / 32], const uint8_t *kbuf, int k0,
                                               bool masked, int sinks) const {
        const int lane = threadIdx.x % 64, half = lane / 32;
        uint32_t gone = 0;
#pragma unroll
        for (int t = 0; t < KT / 32; ++t) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[t][i] = 0.0f;
            const int key = lane % 32;
            const uint8_t *row = kbuf + (t * 32 + key) * DIM * 2;
            const auto add = [&](int x0, int x1) {
#pragma unroll
                for (int d = 0; d < DIM / 16; ++d) {
                    const h8_t k = *(const h8_t *)(row + (((2 * d + half) ^ swz<DIM>(key)) * 16));
#pragma unroll
                    for (int x = 0; x < kParts; ++x) {
                        if (x < x0 || x >= x1) continue;
                        s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[x][d], s[t], 0, 0, 0);
                    }
                }
            };
            add(0, CAREFUL ? 1 : kParts);
            if (CAREFUL) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    gone |= (s[t][i] == -INFINITY ? 1u : 0u) << (16 * t + i);
                asm volatile("" ::: "memory");  // K is read again, not held
                add(1, kParts);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (F32 && (gone >> (16 * t + i) & 1)) s[t][i] = -INFINITY;
            }
        }
        if (masked) {
            asm volatile("; masked tile");  // a branch, not a select in every tile
#pragma unroll
            for (int t = 0; t < KT / 32; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!sees(k0 + t * 32 + 8 * (i / 4) + 4 * half + i % 4, sinks))
                        s[t][i] = -INFINITY;
        }
        return gone;
    }

    // Weights of KT keys as the second product's B operands, 16 keys each.
    template <int KT> struct Weights {
        h8_t w[KT / 16][kWeights];
    };

    // Scores to weights; maximum, sum and what is accumulated so far brought
    // along.  The sum is of the rounded weights, two at a time.
    //
    // The maximum is of scores in powers of two, so that a weight costs one fma
    // and one exponential.  The larger it is, the coarser are the steps of that
    // fma's constant: from 2^23 on a weight may pass binary16's range, or the
    // largest one vanish.  From kFar on (steps of 2^-7) odd() therefore asks for
    // CAREFUL, which takes the difference of the scores themselves first: its m
    // is in their units, until close().
    template <int KT, bool CAREFUL>
    __device__ __forceinline__ void weights(Weights<KT> &out, f16x_t (&s)[KT / 32]) {
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < KT / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
        top = halves_max(top) * (CAREFUL ? 1.0f : c);
        if (__any(top > (CAREFUL ? m : m + kLag))) {
            const float mn = fmaxf(m, top);
            const float f =
                mn == -INFINITY ? 1.0f : factor_of(CAREFUL ? (m - mn) * c : m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] *= f;
        }
        const float base = m == -INFINITY ? 0.0f : CAREFUL ? m : kShift - m;
        const auto power = [&](float x) {
            return CAREFUL ? fmaf(x - base, c, kShift) : fmaf(x, c, base);
        };
        const h2_t ones = {(_Float16)1.0f, (_Float16)1.0f};
#pragma unroll
        for (int b = 0; b < KT / 16; ++b)
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float x0 = __builtin_amdgcn_exp2f(power(s[b / 2][8 * (b % 2) + i]));
                const float x1 = __builtin_amdgcn_exp2f(power(s[b / 2][8 * (b % 2) + i + 1]));
                const h2_t hi = {(_Float16)x0, (_Float16)x1};
                out.w[b][0][i] = hi[0];
                out.w[b][0][i + 1] = hi[1];
                l = __builtin_amdgcn_fdot2(hi, ones, l, false);
                if (FINE) {
                    const h2_t lo = {(_Float16)(x0 - (float)hi[0]), (_Float16)(x1 - (float)hi[1])};
                    out.w[b][kWeights - 1][i] = lo[0];
                    out.w[b][kWeights - 1][i + 1] = lo[1];
                    l = __builtin_amdgcn_fdot2(lo, ones, l, false);
                }
            }
    }

    // The weighted values of the same keys, V in LDS.  CAREFUL: values that are
    // no numbers touch only the rows that see them.
    template <int KT, bool CAREFUL>
    __device__ __forceinline__ void mix(const Weights<KT> &ws, const uint8_t *vbuf, int k0,
                                        int sinks, uint32_t gone) {
        const int lane = threadIdx.x % 64, half = lane / 32;
#pragma unroll
        for (int b = 0; b < KT / 16; ++b) {
            const h8_t *w = ws.w[b];
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
                h8_t v = __builtin_bit_cast(
                    h8_t, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
                if (CAREFUL) {
                    // what is no number leaves the product; rows that see it
                    // are given it afterwards (both signs: NaN).  One whose
                    // score is minus infinity has the weight 0, and 0 times an
                    // infinity is NaN: it counts more than a tile's others.
                    h8_t up, down, see;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float x = (float)v[i];
                        const bool bad = !__builtin_isfinite(x);
                        const bool seen =
                            sees(k0 + 16 * b + 8 * (i / 4) + 4 * half + i % 4, sinks);
                        const bool none = gone >> (8 * b + i) & 1;
                        up[i] = (_Float16)(bad && !(x < 0.0f) ? 1.0f : 0.0f);
                        down[i] = (_Float16)(bad && !(x > 0.0f) ? 1.0f : 0.0f);
                        see[i] = (_Float16)(seen ? none ? 64.0f : 1.0f : 0.0f);
                        if (bad) v[i] = (_Float16)0.0f;
                    }
                    f16x_t zero;
#pragma unroll
                    for (int i = 0; i < 16; ++i) zero[i] = 0.0f;
                    const f16x_t ups =
                        __builtin_amdgcn_mfma_f32_32x32x16_f16(up, see, zero, 0, 0, 0);
                    const f16x_t downs =
                        __builtin_amdgcn_mfma_f32_32x32x16_f16(down, see, zero, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (ups[i] > 0.0f) o[d][i] += INFINITY;
                        if (downs[i] > 0.0f) o[d][i] -= INFINITY;
                        if (fmaxf(ups[i], downs[i]) >= 64.0f) o[d][i] = NAN;
                    }
                }
#pragma unroll
                for (int x = 0; x < kWeights; ++x)
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, w[x], o[d], 0, 0, 0);
            }
        }
    }

    template <int KT, bool CAREFUL>
    __device__ __forceinline__ void step(const uint8_t *kbuf, const uint8_t *vbuf, int k0,
                                         bool masked, int sinks) {
        f16x_t s[KT / 32];
        const uint32_t gone = scores<KT, CAREFUL>(s, kbuf, k0, masked, sinks);
        Weights<KT> ws;
        weights<KT, CAREFUL>(ws, s);
        mix<KT, CAREFUL>(ws, vbuf, k0, sinks, gone);
    }

    // After CAREFUL's tiles: the maximum in powers of two, as without.
    __device__ __forceinline__ void close() { m *= c; }

    // Whether a product met something that is no number, or a maximum lies so far
    // from 0 that the weights have lost their last bits.
    __device__ __forceinline__ bool odd() const {
        if (fabsf(m) >= kFar && m != -INFINITY) return true;
        float z = l * 0.0f;
#pragma unroll
        for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) z += o[d][i] * 0.0f;
        return !(z == 0.0f);
    }
};

// ---- many rows: waves of 32 rows share each key tile ------------------------
// RW waves of 32 rows work on one key tile; KW such groups take every KW-th
// tile each and are joined through LDS at the end.  Two stages of KT keys to a
// group: while its waves work on one, the copies of the next are in flight.
// RW = 4, KW = 1 reads a key least often; RW = 2, KW = 4 (or 2) keeps the
// device busy when there are few rows.
//
// Two prompts of 5001 and 3146 tokens, 32 + 8 heads of 128, binary16: 320 to 340 us,
// 0.84 to 0.89 PFLOP/s, where the library's 8192-cubed product reaches 1.19 on
// this part (float32: twice the products, 545 us).
// Matrix, vector and LDS work are about as long as each other (per 64 keys and
// SIMD 2048, 2000 and 2048 to 2800 cycles of 4300), and the clock falls to
// about 1.7 GHz under them: eight waves in two groups that take turns at matrix
// and vector work, or fragments requested further ahead, cut the cycles and
// not the time.
template <int DIM, int RW, int KW> struct Pass {
    static constexpr int KT = KW > 1 || DIM > 128 ? 32 : 64;
    static constexpr int kTile = KT * DIM * 2;
    static constexpr int kPitch = DIM + 4, kShare = 32 * kPitch * 4;
    static constexpr int kStages = KW * 4 * kTile;
    static constexpr int kLds = KW > 1 && RW * KW * kShare > kStages ? RW * KW * kShare : kStages;
    static constexpr int kThreads = 64 * RW * KW;
    // two workgroups to a compute unit, or eight waves
    static constexpr int kWavesPerSimd = DIM > 128 ? 1 : 2;
};

template <int DIM, bool F32, int RW, int KW, bool CAREFUL>
__device__ __forceinline__ void pass_loop(Rows<DIM, F32, F32> &w, Filler<DIM, false> &f,
                                          const Reach<Pass<DIM, RW, KW>::KT> &r, int t0, int t1,
                                          int top_lo, uint8_t *lds) {
    using P = Pass<DIM, RW, KW>;
    constexpr int KT = P::KT, kTile = P::kTile, kGroups = KT / 16;
    constexpr bool kBoth = RW <= kGroups;  // a wave copies K and V of its keys, or one of them
    constexpr int kMine = kBoth ? kGroups / RW : 1;
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int rw = wave % RW;
    uint8_t *mine = lds + wave / RW * 4 * kTile;
    const int at = 16 * (kBoth ? rw * kMine : rw % kGroups);
    t0 += wave / RW;
    const int count = (t1 - t0 + KW - 1) / KW;  // this group's tiles
    int looked[kMine];
    const auto fill = [&](int i) {
        if (i % 64 == 0) {
            const int key = r.key(min(t0 + (i + lane) * KW, t1 - 1)) + at;
#pragma unroll
            for (int x = 0; x < kMine; ++x) looked[x] = f.look(key + 16 * x);
        }
        const int k = r.key(t0 + i * KW) + at;
        uint8_t *dst = mine + (i & 1) * 2 * kTile + at * DIM * 2;
#pragma unroll
        for (int x = 0; x < kMine; ++x) {
            const int page = __builtin_amdgcn_readlane(looked[x], i % 64);
            uint8_t *d = dst + 16 * x * DIM * 2;
            if (kBoth) {
                f.fill(r, page, k + 16 * x, d, false);
                f.fill(r, page, k + 16 * x, d + kTile, true);
            } else {
                f.fill(r, page, k, d + (rw < kGroups ? 0 : kTile), rw >= kGroups);
            }
        }
    };
    if (count > 0) fill(0);
    // every group goes through as many barriers as the first
    const int rounds = uniform((t1 - t0 + wave / RW + KW - 1) / KW);
    for (int i = 0; i < rounds; ++i) {
        Q4_WAIT_VMCNT(0);
        __syncthreads();
        if (i + 1 < count) fill(i + 1);
        if (i >= count) continue;
        const int k = r.key(t0 + i * KW);
        const uint8_t *kbuf = mine + (i & 1) * 2 * kTile;
        w.template step<KT, CAREFUL>(kbuf, kbuf + kTile, k, CAREFUL || !r.all(k, KT, top_lo),
                                     r.sinks);
    }
}

template <int DIM, bool F32, int RW, int KW>
__global__ __launch_bounds__((Pass<DIM, RW, KW>::kThreads),
                             (Pass<DIM, RW, KW>::kWavesPerSimd)) void pass_kernel(AttentionArgs a,
                                                                                  Plan pl,
                                                                                  int base) {
    using P = Pass<DIM, RW, KW>;
    __shared__ __align__(1024) uint8_t lds[P::kLds];
    __shared__ float ml[2][KW][32 * RW];
    constexpr int R = 32 * RW;
    const int hk = blockIdx.x, split = blockIdx.y;
    Place at = find_tile<R>(a, pl.group, base + blockIdx.z);
    const int count = (at.rows + R - 1) / R;
    if (at.tile < 0 || at.tile >= count) return;
    at.tile = count - 1 - at.tile;  // the tiles with the most keys first
    const int position0 = at.kv - at.rows / pl.group;
    const int row0 = at.tile * R, row1 = min(row0 + R, at.rows);
    const int p0 = position(a, position0, row0 / pl.group);
    const int p1 = position(a, position0, (row1 - 1) / pl.group);
    const Reach<P::KT> r(a, p0, p1);
    const int top_lo = a.window && p1 >= a.window ? p1 - a.window + 1 : 0;
    const int per = max((r.tiles + pl.splits - 1) / pl.splits, pl.least);
    const int t0 = min(split * per, r.tiles), t1 = min(t0 + per, r.tiles);
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int mine = wave % RW * 32 + lane % 32, row = row0 + mine;
    Rows<DIM, F32, F32> w;
    {
        typename Rows<DIM, F32, F32>::Raw raw;
        w.request(raw, a, at, pl.group, hk, row, position0);
        w.take(raw);
    }
    if (t0 < t1) {
        Filler<DIM, false> f(a, at.s, hk);
        pass_loop<DIM, F32, RW, KW, false>(w, f, r, t0, t1, top_lo, lds);
        if (__builtin_expect(__syncthreads_or(w.odd()), 0)) {
            w.clear();
            pass_loop<DIM, F32, RW, KW, true>(w, f, r, t0, t1, top_lo, lds);
            w.close();
        }
    }
    float l = halves_sum(w.l), m = w.m;
    const int half = lane / 32;
    if (KW > 1) {
        // join the groups: the first takes over its rows' sum
        if (lane < 32) ml[0][wave / RW][mine] = m, ml[1][wave / RW][mine] = l;
        __syncthreads();
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < KW; ++i) top = fmaxf(top, ml[0][i][mine]);
        const float zero = top == -INFINITY ? 0.0f : top;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < KW; ++i) l += ml[1][i][mine] * factor_of(ml[0][i][mine] - zero);
        const float fs = factor_of(m - zero);
        m = top;
        float *share = (float *)(lds + wave * P::kShare) + (lane % 32) * P::kPitch + 4 * half;
#pragma unroll
        for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                f4_t v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = w.o[d][i + e] * fs;
                *(f4_t *)(share + 32 * d + 2 * i) = v;
            }
        __syncthreads();
        if (pl.splits > 1 && wave < RW && lane < 32 && row < row1) {
            const int64_t out = (int64_t)(at.first + row / pl.group) * a.q_heads +
                                hk * pl.group + row % pl.group;
            put_ml(a, pl, split, out, m, l);
        }
        if (wave < RW && lane < 32) ml[1][0][mine] = l;
        __syncthreads();
        if (pl.splits > 1 && t0 >= t1) return;
        for (int e = threadIdx.x; e < (row1 - row0) * (DIM / 4); e += P::kThreads) {
            const int rr = e / (DIM / 4), d = e % (DIM / 4) * 4;
            const float *src = (const float *)(lds + rr / 32 * P::kShare) + rr % 32 * P::kPitch + d;
            f4_t o = *(const f4_t *)src;
#pragma unroll
            for (int i = 1; i < KW; ++i) {
                const f4_t v = *(const f4_t *)(src + i * RW * P::kShare / 4);
#pragma unroll
                for (int x = 0; x < 4; ++x) o[x] += v[x];
            }
            const int token = (row0 + rr) / pl.group;
            const int64_t out = (int64_t)(at.first + token) * a.q_heads + hk * pl.group +
                                (row0 + rr) % pl.group;
            put4<F32>(a, pl, split, out, DIM, d, o, ml[1][0][rr], position0 + token >= 0);
        }
        return;
    }
    if (row >= row1) return;
    const int64_t out = (int64_t)(at.first + row / pl.group) * a.q_heads + hk * pl.group +
                        row % pl.group;
    // (one wave group: 128-row tiles, whose key axis is never split)
#pragma unroll
    for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            put_y4<F32>(a, out, DIM, 32 * d + 2 * i + 4 * half,
                        f4_t{w.o[d][i], w.o[d][i + 1], w.o[d][i + 2], w.o[d][i + 3]}, l,
                        w.p >= 0);
}

// ---- few rows: every wave streams its own keys for the same 32 rows ---------
// No barrier in the loop: a wave fills its own K and V tile and waits for its
// own copies.  One tile each, not two stages: K is requested again as soon as
// the scores are formed, V as soon as it is mixed, and the other waves of the
// workgroup cover what that leaves open, so nearly all of LDS is in flight.
// The waves' results are joined through LDS at the end.
//
// Bound by the bytes of K and V: one conversation of 131071 keys (32 + 8 heads of
// 128) in 83 us, 6.5 TB/s, and 5 us for joining its parts, where a plain
// streaming read of 512 MiB reaches 7.1.
constexpr int kStepRows = 32, kStepKeys = 32;

template <int DIM, bool F32, bool CAREFUL>
__device__ __forceinline__ void step_loop(Rows<DIM, F32, true> &w, Filler<DIM, true> &f,
                                          const Reach<kStepKeys> &r, int t, int t1, int stride,
                                          int top_lo, uint8_t *kbuf, int look0,
                                          int look1, bool started) {
    constexpr int KT = kStepKeys;
    constexpr int kCopies = KT / 16 * Filler<DIM, true>::kCopies;  // of K, or of V
    constexpr int kHalf = 16 * DIM * 2;
    uint8_t *vbuf = kbuf + 2 * kHalf;
    const int lane = threadIdx.x % 64;
    if (t >= t1) return;
    int i = 0;  // the tile's lane in look0 and look1
    int page0 = __builtin_amdgcn_readlane(look0, 0), page1 = __builtin_amdgcn_readlane(look1, 0);
    bool counted = false;  // the copies requested last are all kCopies of them
    if (!started) {
        const int k = r.key(t);
        f.fill(r, page0, k, kbuf, false);
        f.fill(r, page1, k + 16, kbuf + kHalf, false);
        f.fill(r, page0, k, vbuf, true);
        f.fill(r, page1, k + 16, vbuf + kHalf, true);
    }
    for (; t < t1; t += stride) {
        const int k = r.key(t), next = r.key(t + stride);
        const bool more = t + stride < t1;
        f16x_t s[KT / 32];
        // outstanding: K, then V
        if (counted)
            Q4_WAIT_VMCNT(kCopies);
        else
            Q4_WAIT_VMCNT(0);
        Q4_WAIT_LGKM0();
        asm volatile("" ::: "memory");
        const uint32_t gone = w.template scores<KT, CAREFUL>(
            s, kbuf, k, CAREFUL || !r.all(k, KT, top_lo), r.sinks);
        Q4_WAIT_LGKM0();
        asm volatile("" ::: "memory");
        counted = false;
        if (more) {
            i = (i + 1) % 64;
            if (__builtin_expect(i == 0, 0)) {
                const int mine = r.key(min(t + stride + lane * stride, t1 - 1));
                look0 = f.look(mine);
                look1 = f.look(mine + 16);
            }
            page0 = __builtin_amdgcn_readlane(look0, i);
            page1 = __builtin_amdgcn_readlane(look1, i);
            counted = f.fill(r, page0, next, kbuf, false);
            counted &= f.fill(r, page1, next + 16, kbuf + kHalf, false);
        }
        typename Rows<DIM, F32, true>::template Weights<KT> ws;
        w.template weights<KT, CAREFUL>(ws, s);
        // outstanding: V, then the next K
        if (counted)
            Q4_WAIT_VMCNT(kCopies);
        else
            Q4_WAIT_VMCNT(0);
        asm volatile("" ::: "memory");
        w.template mix<KT, CAREFUL>(ws, vbuf, k, r.sinks, gone);
        Q4_WAIT_LGKM0();
        asm volatile("" ::: "memory");
        if (more) {
            counted = f.fill(r, page0, next, vbuf, true);
            counted &= f.fill(r, page1, next + 16, vbuf + kHalf, true);
        }
    }
}

// (two waves to a SIMD: a second workgroup of four, or one of eight)
template <int DIM, bool F32, int W>
__global__ __launch_bounds__(64 * W, DIM > 128 ? 1 : 2) void step_kernel(AttentionArgs a, Plan pl,
                                                                         int base) {
    constexpr int KT = kStepKeys;
    constexpr int kHalf = 16 * DIM * 2;
    constexpr int kPitch = DIM + 4;
    // a wave's K and V tiles, later its rows
    constexpr int kShare = 32 * kPitch * 4;
    static_assert(4 * kHalf <= kShare && kShare % 256 == 0, "both fit");
    __shared__ __align__(1024) uint8_t lds[W * kShare];
    __shared__ float ml[2][W][32];
    const int hk = blockIdx.x, split = blockIdx.y;
    const Place at = find_tile<kStepRows>(a, pl.group, base + blockIdx.z);
    const int row0 = at.tile * kStepRows;
    if (row0 < 0 || row0 >= at.rows) return;
    const int row1 = min(row0 + kStepRows, at.rows);
    const int position0 = at.kv - at.rows / pl.group;
    const int p0 = position(a, position0, row0 / pl.group);
    const int p1 = position(a, position0, (row1 - 1) / pl.group);
    const Reach<KT> r(a, p0, p1);
    const int top_lo = a.window && p1 >= a.window ? p1 - a.window + 1 : 0;
    const int per = max((r.tiles + pl.splits - 1) / pl.splits, pl.least);
    const int t0 = min(split * per, r.tiles), t1 = min(t0 + per, r.tiles);
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    uint8_t *mine = lds + wave * kShare;
    Filler<DIM, true> f(a, at.s, hk);
    Rows<DIM, F32, true> w;
    const int t = t0 + wave;
    int look0 = -1, look1 = -1;
    {
        typename Rows<DIM, F32, true>::Raw raw;
        if (t < t1) {
            const int k = r.key(min(t + lane * W, t1 - 1));
            look0 = f.look(k);
            look1 = f.look(k + 16);
        }
        w.request(raw, a, at, pl.group, hk, row0 + lane % 32, position0);
        if (t < t1) {
            const int k = r.key(t);
            const int page0 = __builtin_amdgcn_readlane(look0, 0);
            const int page1 = __builtin_amdgcn_readlane(look1, 0);
            f.fill(r, page0, k, mine, false);
            f.fill(r, page1, k + 16, mine + kHalf, false);
            f.fill(r, page0, k, mine + 2 * kHalf, true);
            f.fill(r, page1, k + 16, mine + 3 * kHalf, true);
        }
        w.take(raw);
    }
    step_loop<DIM, F32, false>(w, f, r, t, t1, W, top_lo, mine, look0, look1, true);
    if (__builtin_expect(__any(w.odd()), 0)) {
        w.clear();
        if (t < t1) {
            const int k = r.key(min(t + lane * W, t1 - 1));
            look0 = f.look(k);
            look1 = f.look(k + 16);
        }
        step_loop<DIM, F32, true>(w, f, r, t, t1, W, top_lo, mine, look0, look1, false);
        w.close();
    }
    // join the waves
    w.l = halves_sum(w.l);
    if (lane < 32) ml[0][wave][lane] = w.m, ml[1][wave][lane] = w.l;
    __syncthreads();
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) m = fmaxf(m, ml[0][i][lane % 32]);
    const float fs = factor_of(w.m - (m == -INFINITY ? 0.0f : m));
    if (lane % 32 < row1 - row0) {
        float *mrow = (float *)mine + (lane % 32) * kPitch + 4 * (lane / 32);
#pragma unroll
        for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                f4_t v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = w.o[d][i + e] * fs;
                *(f4_t *)(mrow + 32 * d + 2 * i) = v;
            }
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
            const f4_t v = *(const f4_t *)((const float *)(lds + i * kShare) + rr * kPitch + d);
#pragma unroll
            for (int x = 0; x < 4; ++x) o[x] += v[x];
            l += ml[1][i][rr] * factor_of(ml[0][i][rr] - (m == -INFINITY ? 0.0f : m));
        }
        const int token = (row0 + rr) / pl.group;
        const int64_t out = (int64_t)(at.first + token) * a.q_heads + hk * pl.group +
                            (row0 + rr) % pl.group;
        if (pl.splits > 1 && d == 0) put_ml(a, pl, split, out, m, l);
        if (pl.splits > 1 && t0 >= t1) continue;
        put4<F32>(a, pl, split, out, DIM, d, o, l, position0 + token >= 0);
    }
}

// ---- choices on the host ----------------------------------------------------
struct Choice {
    // rows of a tile: 128 and 64 (waves share the keys, or half of them), 32
    // (every wave on its own keys)
    int rows;
    int waves;  // of a 32-row workgroup
    int64_t tiles;
    int splits;
    int least;  // key tiles of a part, at least
    size_t part, bytes;  // workspace: bytes of the partial rows, and in all
};

// How a call is cut into work items.  The host knows the sizes, not the
// conversations' lengths: those may change between replays of a graph.
Choice choose(const AttentionArgs &a) {
    Choice ch;
    const int dim = a.cache.dim, heads = a.cache.heads;
    const int64_t rows = (int64_t)a.n * (a.q_heads / heads);
    const int64_t cus = device_shape().cus;
    // Up to as many rows to a conversation as a 32-row tile holds, the waves of
    // a workgroup share the rows and split the keys.  With more, they share the
    // keys: 128 rows to a tile if that gives every compute unit one, 64 if not
    // (512 tokens of 4 heads to each of 8 key/value heads, 1100 keys each: 21 us
    // on 64-row tiles; 35 us on 128-row ones, 48 us with their key axis split).
    if (rows <= (int64_t)kStepRows * a.batch)
        ch.rows = 32;
    else
        ch.rows = (rows / 128 + (a.batch + 1) / 2) * heads >= cus ? 128 : 64;
    const int R = ch.rows;
    ch.tiles = rows / R + a.batch;
    // the items that are likely to have work: not all tiles do
    const int64_t likely = (R > 32 ? rows / R + (a.batch + 1) / 2
                                   : (rows / R > a.batch ? rows / R : a.batch)) *
                           heads;
    // the key tiles a row tile can have at most
    const int KT = R == 128 && dim <= 128 ? 64 : 32;
    int64_t keys = (int64_t)a.table_stride << a.cache.page_shift;
    if (a.window) {
        const int64_t near = (int64_t)a.window + a.sinks + 2 * R + 2 * KT;
        if (near < keys) keys = near;
    }
    const int64_t most = (keys + KT - 1) / KT;
    int64_t splits;
    ch.waves = dim > 128 ? 2 : 4;
    if (R > 32) {
        splits = cus / likely;  // (128-row tiles are taken where that is one at most)
        ch.least = 16;
    } else {
        // workgroups that run at once: two to a compute unit, four of 64-wide heads
        const int64_t slots = cus * (dim > 64 ? 2 : 4);
        // One conversation: as many parts as run at once.  Several are of
        // several lengths: more, so that the long ones do not end alone, but of
        // 1024 keys at least (a part costs about 4 us beside its keys), or of
        // what gives every slot one where there are fewer.  64 conversations of
        // 400 to 8192 keys, joining included: 209 us unsplit, 187 us so, 203 us
        // in parts of 512; 32 of 4096 keys of 256: 95 us in three parts, 94 us
        // in four, 105 us in eight; 2 of 1700 keys: 17 us unsplit, 10 us in
        // parts of 256.  Parts of 512, 1024 and 2048 keys elsewhere (us): 4 of
        // 32768 keys 87, 83 and 81; 16 of 1600 to 32768 193, 193 and 198; 32 of
        // 16384 (heads of 256) 213, 224 and 216; 128 of 100 to 2048 104, 117 and
        // 100; 128 of 400 to 8192 (heads of 64) 181, 180 and 211.
        splits = ((a.batch == 1 ? 1 : 4) * slots + (a.batch == 1 ? 0 : likely - 1)) / likely;
        const int64_t fair = (most * likely + slots - 1) / slots;
        ch.least = fair > 32 ? 32 : fair < 2 * ch.waves ? 2 * ch.waves : (int)fair;
        // too few keys to split: the workgroup's own waves take them, eight
        // (four) instead of four (two) while there are units to spare
        if (most / ch.least < 2 && likely <= cus) ch.waves *= 2;
    }
    if (splits > most / ch.least) splits = most / ch.least;
    if (splits > kMaxSplits) splits = kMaxSplits;
    const int64_t out = (int64_t)a.n * a.q_heads;
    const int64_t room = (int64_t)kWorkspaceBytes / (out * (dim + 2) * 4);
    if (splits > room) splits = room;
    ch.splits = splits < 2 ? 1 : (int)splits;
    if (ch.splits == 1) ch.least = 1;
    ch.part = ch.splits > 1 ? (size_t)ch.splits * (size_t)out * (size_t)dim * 4u : 0;
    ch.bytes = ch.splits > 1 ? ch.part + (size_t)ch.splits * (size_t)out * 8u : 0;
    return ch;
}

template <int DIM, bool F32>
hipError_t run(const AttentionArgs &a, const Choice &ch, const Plan &pl, hipStream_t stream) {
    constexpr int W = DIM > 128 ? 2 : 4;
    // heads fastest: the tiles of one head of a conversation come to the same
    // die, eight heads to eight dies, and share its L2
    for (int64_t base = 0; base < ch.tiles; base += 65535) {
        const int64_t tiles = ch.tiles - base < 65535 ? ch.tiles - base : 65535;
        const dim3 grid((uint32_t)a.cache.heads, (uint32_t)ch.splits, (uint32_t)tiles);
        if (ch.rows == 128)
            hipLaunchKernelGGL((pass_kernel<DIM, F32, 4, 1>), grid, dim3(256), 0, stream, a, pl,
                               (int)base);
        else if (ch.rows == 64)
            hipLaunchKernelGGL((pass_kernel<DIM, F32, 2, W>), grid, dim3(128 * W), 0, stream, a,
                               pl, (int)base);
        else if (ch.waves == W)
            hipLaunchKernelGGL((step_kernel<DIM, F32, W>), grid, dim3(64 * W), 0, stream, a, pl,
                               (int)base);
        else
            hipLaunchKernelGGL((step_kernel<DIM, F32, 2 * W>), grid, dim3(128 * W), 0, stream, a,
                               pl, (int)base);
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

int attention_tile_rows(const AttentionArgs &a) { return choose(a).rows; }

hipError_t launch_attention(const AttentionArgs &a, int x_f16, void *ws, hipStream_t stream) {
    const Choice ch = choose(a);
    const Plan pl = {a.q_heads / a.cache.heads, ch.splits, ch.least, (float *)ws,
                     (float *)((uint8_t *)ws + ch.part)};
    return x_f16 ? by_dim<false>(a, ch, pl, stream) : by_dim<true>(a, ch, pl, stream);
}

}  // namespace q4
