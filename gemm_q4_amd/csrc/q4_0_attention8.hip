// Attention of a ragged batch over a paged cache of 8-bit codes.
//
//     y = sum_j softmax_j(scale q . s_j c_j) t_j e_j
//
// with codes c, e of K and V (integers from -128 to 127) and one float32 scale
// s, t to a row of either.  The codes are binary16 numbers exactly, so both
// products run on the binary16 matrix cores without a rounding of K or V; a
// key's scale multiplies its score, and a value's scale its weight, in float32.
//
// Codes to binary16: with the sign bit flipped a code c is the byte c + 128, which
// under the exponent byte 0x64 reads as 1024 + 128 + c; one packed subtraction
// leaves c.  Five instructions for four codes.
//
// A value's weight is p t with p = exp(x - m) in float32, which enters its product in
// binary16 parts.  While all scales t of a wave's keys lie within some powers of two, t
// is brought to the largest met so far (a power of two, so without rounding) before it
// is multiplied; that running exponent is lifted, and what is accumulated rescaled,
// like the maximum of the softmax.  A row's strongest key then has a weight that
// binary16 holds in full.  Where a tile's scales lie further apart than that (a token
// whose values are a thousand times another's, seen by other rows of the tile, or with
// next to no weight) the tile is done again with an exponent of its own for every row, of
// the largest p t among the keys it sees: in blocks of 16 rows, by code apart, so that
// the usual loops have none of its instructions and registers.  The scales of keys that
// no row of a tile sees are taken as 0 and their codes are finite whatever they are, so
// what a page holds past its conversation's end never meets the arithmetic.  (One key
// half way with a scale 2^12 below the others': 64 conversations 191 us instead of 101,
// prompts 1075 instead of 321.)
//
// A score is formed less the running maximum, by one fused operation on its product:
// scores of any size lose nothing, and while the maximum holds its exponential
// follows at once.  Scores of binary16 rows are in powers of two (K's scales carry
// the factor, the same for all rows); float32 rows have a factor `c` of their own.
//
// Measured (32 + 8 heads of 128, binary16 rows but for the first; rates of the bytes or
// operations that the call cannot do without): one conversation of 448 keys 9.2 us, a
// chain of lengths, page table, keys and the join of the waves; of 131072 keys 52 us, 5.3
// TB/s (over binary16 91 us); 64 conversations of 470 to 8192 keys, one to four tokens
// each, 100 us, 5.8 TB/s (185 us over binary16 with a token each); the last 2438 of 5001
// tokens beside a prompt of 3146 321 us, 722 TFLOP/s.
#include "q4_0_attention.h"
#include "q4_0_dma.h"

namespace q4 {

namespace {

typedef int i2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i2_t *lds_i2_t;

// Four codes as two pairs of binary16.
__device__ __forceinline__ void codes4(uint32_t w, uint32_t &h0, uint32_t &h1) {
    const uint32_t top = 0x64646464u, b = w ^ 0x80808080u;
    const h2_t off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
    h0 = as_u32(as_h2(__builtin_amdgcn_perm(top, b, 0x04010400u)) + off);
    h1 = as_u32(as_h2(__builtin_amdgcn_perm(top, b, 0x04030402u)) + off);
}
__device__ __forceinline__ h8_t codes8(uint32_t w0, uint32_t w1) {
    uint32_t h[4];
    codes4(w0, h[0], h[1]);
    codes4(w1, h[2], h[3]);
    return pack_h8(h);
}

// Direct copy of 4 bytes per lane into LDS: lane i's at lds + 4 i.
__device__ __forceinline__ void dma4(const void *src, uint8_t *lds) {
    const uint32_t base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
                 :
                 : "v"(src), "s"(base)
                 : "memory", "m0");
}

static __device__ const uint32_t kNanWord = 0x7FC00000u;

// A launch's arguments; `base`: the first of its tiles.
struct Call {
    AttentionArgs a;
    Plan pl;
    int base;
};
// They once more, from memory: a rare path that took them from the kernel's own would
// keep registers for them through the usual one.
__device__ __forceinline__ const Call &call_again() {
    auto p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const Call *)p;
}

// x of the four lanes l, l + 16, l + 32, l + 48 joined.
template <typename F> __device__ __forceinline__ float quads(float x, F f) {
    uint32_t u = __builtin_bit_cast(uint32_t, x);
    auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    x = f(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
    u = __builtin_bit_cast(uint32_t, x);
    r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return f(__builtin_bit_cast(float, (uint32_t)r[0]),
             __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float quads_max(float x) {
    return quads(x, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float quads_sum(float x) {
    return quads(x, [](float a, float b) { return a + b; });
}

// The exponent that brings a scale into [1/2, 1); far below any for 0 and for
// what is no number.
constexpr int kNoExponent = -1000;
// The same where exponents are compared with maxima of scores: below any of those too.
constexpr float kNever = 1e6f;
// Powers of two that the scales of a row's keys may lie apart for one exponent to do.
// The strongest key's weight is then 2^(kShift - 1 - kSpread) or more, where half a step
// of the least numbers is 2^-25.
constexpr int kSpread = 10;
__device__ __forceinline__ int exponent(float t) {
    const float a = fabsf(t);
    return a > 0.0f && a <= FLT_MAX ? __builtin_amdgcn_frexp_expf(a) : kNoExponent;
}
template <int CTRL> __device__ __forceinline__ int turned_max(int x) {
    return max(x, __builtin_amdgcn_mov_dpp(x, CTRL, 0xF, 0xF, true));
}
// By lane moves alone: LDS permutes would be a chain of six latencies.
__device__ __forceinline__ int wave_max(int x) {
    x = turned_max<0x121>(x);  // within 16 lanes, turned by one, two, four, eight
    x = turned_max<0x122>(x);
    x = turned_max<0x124>(x);
    x = turned_max<0x128>(x);
    auto r = __builtin_amdgcn_permlane16_swap((uint32_t)x, (uint32_t)x, false, false);
    x = max((int)r[0], (int)r[1]);
    r = __builtin_amdgcn_permlane32_swap((uint32_t)x, (uint32_t)x, false, false);
    return uniform(max((int)r[0], (int)r[1]));
}
// A value's scale, relative to 2^top; one that is infinite is no number either.
__device__ __forceinline__ float number(float t) { return fabsf(t) <= FLT_MAX ? t : NAN; }
__device__ __forceinline__ float relative(float t, int top, int shift) {
    return __builtin_amdgcn_ldexpf(number(t), shift - top);
}

// The exponents of the scales that a wave has met: the largest and the smallest.
struct Span8 {
    int top = kNoExponent, low = -kNoExponent;
    __device__ __forceinline__ bool apart() const { return top - low > kSpread; }
    // `mine` (this lane's scale; by all lanes) taken in: whether that changed them.
    __device__ __forceinline__ bool take(float mine) {
        const int e = exponent(mine);
        if (!__any(e > top || (e != kNoExponent && e < low))) return false;
        top = max(wave_max(e), top);
        low = min(-wave_max(e == kNoExponent ? e : -e), low);
        return true;
    }
};

// A row's own exponent as the ceiling of `ref`, the power of two of the largest weight
// (p t) that the row has met, relative to its maximum of the softmax.
__device__ __forceinline__ int own_exponent(float ref) { return (int)ceilf(ref); }
// p times the mantissa of the scale t, and the power of two of p t (none for 0, and for
// what is no number).
__device__ __forceinline__ float mantissa(float p, float t) {
    return p * __builtin_amdgcn_frexp_mantf(t);
}
__device__ __forceinline__ float power(float z, float t) {
    return fabsf(z) > 0.0f ? (float)(__builtin_amdgcn_frexp_expf(z) + __builtin_amdgcn_frexp_expf(t))
                           : -kNever;
}
// `ref` after the maximum rose by `u` powers of two and a tile's largest weight is 2^most;
// what is accumulated is multiplied by the result (less than 4, 0 for what has vanished).
__device__ __forceinline__ float lifted_to(float &ref, float u, float most) {
    const int was = own_exponent(ref);
    ref = fmaxf(fmaxf(ref - u, most), -kNever);
    return __builtin_amdgcn_exp2f((float)(was - own_exponent(ref)) - u);
}

// Sums that took in many tiles: a faint weight's share would vanish in them (each is off
// by half a step of the sum, and of 10^5 keys beside a strong one most would be lost).
// So every kFold tiles of a wave, if half as many are left, they are put aside, in memory:
// registers are few, and the way there is rare.  144 tokens of 89120 keys, float32:
// off by 5e-7 so, by 3e-5 without; 320 of 131072 with heads of 256, 1024 tiles to a
// wave, beside a strong key by 1.5e-5 and by 2.2e-4.  It takes 2 to 6% of such calls' time
// (128 conversations of 131072 keys 5.48 ms instead of 5.17).  Every 32 tiles, passes over
// 5000 keys would take 343 us instead of 316.
constexpr int kFold = 64;
typedef volatile __attribute__((address_space(5))) f4_t *private_f4_t;
template <typename W> struct Total {
    f4_t o[W::kQuads];
    float l, m;
    int top;
    bool seen;
    // now: the exponent of the sums; more: some were put aside before.
    __device__ __forceinline__ void fold(W &w, int now, bool more) {
        if (more) back(w, now);
        const private_f4_t at = (private_f4_t)o;
#pragma unroll
        for (int i = 0; i < W::kQuads; ++i) at[i] = w.quad(i);
        l = w.l, m = w.m, top = now, seen = w.over != -INFINITY;
        w.l = 0.0f;
        w.zero();
    }
    // What was put aside, brought to the maximum and the exponent now and added again.
    __device__ __forceinline__ void back(W &w, int now) {
        const float down = (m - w.m) * w.c;
        const float f = seen ? __builtin_amdgcn_exp2f((float)(top - now) + down) : 0.0f;
        if (seen) w.l += l * factor_of(down);
        const private_f4_t at = (private_f4_t)o;
#pragma unroll
        for (int i = 0; i < W::kQuads; ++i) w.add(i, at[i], f);
    }
};

// The cache as a tile's loads see it: head hk of the pages of conversation s.
struct Source {
    const uint8_t *k, *v;  // codes of this head on page 0
    const float *ks, *vs;  // scales, likewise
    const int32_t *table;
    int64_t page_rows;  // rows of all heads of a page
    int pages, table_stride, shift;
    __device__ __forceinline__ Source(const AttentionArgs &a, int s, int hk)
        : table(a.table + (int64_t)s * a.table_stride),
          page_rows((int64_t)a.cache.heads << a.cache.page_shift), pages((int)a.cache.pages),
          table_stride(a.table_stride), shift(a.cache.page_shift) {
        const int64_t row = (int64_t)hk << shift;
        k = (const uint8_t *)a.cache.k + row * a.cache.dim;
        v = (const uint8_t *)a.cache.v + row * a.cache.dim;
        ks = a.cache.k_scale + row;
        vs = a.cache.v_scale + row;
    }
    // The page of key `key` (of the lane's own choice), -1 if it has none.
    __device__ __forceinline__ int look(int key) const {
        const int slot = key >> shift;
        const int page = slot < table_stride ? table[slot] : -1;
        return page < pages ? max(page, -1) : -1;
    }
    // Row of `key` on `page`.  A key without a page is given a row of page 0,
    // whose codes do no harm: its scales say what it is.
    __device__ __forceinline__ int64_t row(int page, int key) const {
        return max(page, 0) * page_rows + (key & ((1 << shift) - 1));
    }
    // Where the scale of `key` is read: 0 for one that no row of the tile sees;
    // without a page K's is NaN.
    template <int KT>
    __device__ __forceinline__ const void *scale(const Reach<KT> &r, int page, int key,
                                                 bool is_v) const {
        const void *p = (is_v ? vs : ks) + row(page, key);
        if (page < 0) p = is_v ? (const void *)&kZeroPiece : (const void *)&kNanWord;
        return r.any(key) ? p : (const void *)&kZeroPiece;
    }
};

// ---- few rows: every wave streams its own keys ------------------------------
// A wave works on tiles of 64 keys and one or two blocks of 16 rows, with
// v_mfma_f32_16x16x32_f16: S^T = K Q^T leaves row l % 16's scores of the keys
// 16 b + 4 (l / 16) + 0..3 in lane l, and the weights of two such blocks are as they
// lie the B operand of O^T = V^T P^T, whose A operand (eight keys of one column
// to a lane) the transposing 8-bit LDS read delivers from row-major V.
//
// Bound by the bytes: 6 to 6.7 TB/s while the keys stream.  What keeps a call from that
// as a whole is the chain before the first key (4 to 5 us), the join (5 us), and, with
// conversations of several lengths, the slots that end early: the longest come first.  64 keys a tile: the
// scales of 64 are one copy of 4 bytes to a lane.  Up to 32 rows: 64 rows to a wave
// (which leaves one wave to a SIMD) took 200 instead of 158 us for 16 conversations
// of 8192 keys, eight tokens of 8 heads each.
constexpr int kStepRows = 32, kStepKeys = 64;

// Codes in LDS are rows of DIM bytes, their 16-byte pieces XOR-swizzled: sixteen
// neighbouring keys at one piece, and keys 8 h + 0..7 with 16 + 8 h + 0..7 at one
// piece, fall on distinct banks.
template <int DIM> __device__ __forceinline__ int swz8(int key) {
    constexpr int kLow = DIM == 256 ? 0 : DIM == 128 ? 1 : 2;  // rows of 256 bytes, as a power
    return ((key >> kLow) & ((1 << (3 - kLow)) - 1)) |
           ((((key >> 3) ^ (key >> 4)) & 1) << (3 - kLow));
}

// Copies of a tile into a wave's share of LDS: codes of K, of V, then scales of
// K, of V.  Always as many of them, whatever the keys are.
template <int DIM> struct StepFiller : Source {
    static constexpr int kCopies = DIM / 64;  // of 16 rows, 1 KB each
    static constexpr int kAll = kStepKeys / 16 * kCopies + 1;  // a tile's, of K or of V
    static constexpr int kCodes = kStepKeys * DIM;
    const int lane;
    uint32_t off[2][kCopies];
    __device__ __forceinline__ StepFiller(const AttentionArgs &a, int s, int hk, int lane_)
        : Source(a, s, hk), lane(lane_) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int j = 0; j < kCopies; ++j) {
                const int row = j * (1024 / DIM) + lane / (DIM / 16);
                off[g][j] = row * DIM + ((lane % (DIM / 16)) ^ swz8<DIM>(16 * g + row)) * 16;
            }
    }
    // ONCE: no other tile reads these keys, and the copies carry the non-temporal hint.
    template <bool ONCE>
    __device__ __forceinline__ void fill(const Reach<kStepKeys> &r, const int (&page)[4], int key,
                                         uint8_t *lds, bool is_v) const {
        uint8_t *dst = lds + (is_v ? kCodes : 0);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const uint8_t *src = (is_v ? v : k) + row(page[g], key + 16 * g) * DIM;
#pragma unroll
            for (int j = 0; j < kCopies; ++j) {
                if (ONCE)
                    dma16_once_at(src, off[g & 1][j], dst + g * 16 * DIM + j * 1024);
                else
                    dma16_at(src, off[g & 1][j], dst + g * 16 * DIM + j * 1024);
            }
        }
        // the lane's own page, chosen among copies (an identity move): the pages
        // themselves stay in scalar registers, as the copies' bases have to
        const auto copy = [](int x) { return __builtin_amdgcn_mov_dpp(x, 0xE4, 0xF, 0xF, true); };
        const int p0 = copy(page[0]), p1 = copy(page[1]), p2 = copy(page[2]), p3 = copy(page[3]);
        const int mine = lane < 32 ? (lane < 16 ? p0 : p1) : (lane < 48 ? p2 : p3);
        dma4(scale(r, mine, key + lane, is_v),
             lds + 2 * kCodes + (is_v ? kStepKeys * 4 : 0));
    }
};

// A block of 16 rows: queries, running maximum (of scores without `c`; 0 before the
// first), sum (this lane's keys) and unnormalised result.  A score above the maximum
// by more than `over` lifts it (any does, the first time).  Weights are held in two
// binary16 parts, as 2^kShift of the largest: what is lost of one is 2^-28 of the row's
// strongest key's or less, 2^-38 with the row's own exponent, `ref`.
template <int DIM, bool F32> struct Block {
    static constexpr int kParts = F32 ? 2 : 1;  // of q
    static constexpr float kLag = 1.0f;
    static constexpr int kShift = 14;
    h8_t q[kParts][DIM / 32];
    f4_t o[DIM / 16];
    float m, l, c, over, ref;
    int p, lo;

    struct Raw {
        u4_t x[kParts * DIM / 32];
    };
    // Row r (of the conversation's `rows`); rows past the end repeat the last.
    // Lane l holds elements 64 j + 16 (l / 16) + 0..15 of row l % 16.
    __device__ __forceinline__ void request(Raw &raw, const AttentionArgs &a, const Place &pl,
                                            int group, int hk, int r, int position0, int g) {
        const int rr = min(r, pl.rows - 1);
        const int token = rr / group;
        p = position(a, position0, token);
        lo = a.window && p >= a.window ? p - a.window + 1 : 0;
        c = F32 ? finite(a.scale * kLog2e) : 1.0f;
        const int64_t at = (int64_t)(pl.first + token) * a.q_stride +
                           (int64_t)(hk * group + rr % group) * DIM + 16 * g;
        const u4_t *src = (const u4_t *)((const uint8_t *)a.q + at * (F32 ? 4 : 2));
#pragma unroll
        for (int j = 0; j < DIM / 64; ++j)
#pragma unroll
            for (int x = 0; x < 2 * kParts; ++x)
                raw.x[j * 2 * kParts + x] = src[j * (F32 ? 16 : 8) + x];
    }
    __device__ __forceinline__ void clear() {
        m = 0.0f;
        over = -INFINITY;
        ref = -kNever;
        l = 0.0f;
        zero();
    }
    __device__ __forceinline__ void take(const Raw &raw) {
        if (!F32) {
#pragma unroll
            for (int d = 0; d < DIM / 32; ++d) q[0][d] = __builtin_bit_cast(h8_t, raw.x[d]);
            return;
        }
        // the row's largest element brought into [1/2, 1), so that its parts are
        // neither infinite nor faint whatever q's magnitude
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < kParts * DIM / 8; ++i) {
            const uint32_t bits = raw.x[i / 4][i % 4];
            top = fmaxf(top, fabsf(__builtin_bit_cast(float, bits)));
        }
        const int e = __builtin_amdgcn_frexp_expf(quads_max(top));
        c = finite(__builtin_amdgcn_ldexpf(c, e));
#pragma unroll
        for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t bits = raw.x[(d * kParts + i / 4) % (kParts * DIM / 32)][i % 4];
                const float v = __builtin_amdgcn_ldexpf(__builtin_bit_cast(float, bits), -e);
                const _Float16 hi = (_Float16)v;
                q[0][d][i] = hi;
                q[kParts - 1][d][i] = (_Float16)(v - (float)hi);
            }
    }
    __device__ __forceinline__ bool sees(int key, int sinks) const {
        return key <= p && (key >= lo || key < sinks);
    }
    static constexpr int kQuads = DIM / 16;  // of o
    __device__ __forceinline__ f4_t quad(int i) const { return o[i]; }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int d = 0; d < DIM / 16; ++d) o[d] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __device__ __forceinline__ void add(int i, f4_t x, float f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = fmaf(x[e], f, o[i][e]);
    }
    __device__ __forceinline__ void rescale(float f) {
#pragma unroll
        for (int d = 0; d < DIM / 16; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[d][i] *= f;
    }
    // Scores of 64 keys, less the maximum, to weights; the maximum brought along.  By how
    // many powers of two it rose; APART: `o` is yet to fall by as much.
    template <bool APART> __device__ __forceinline__ float soften(f4_t (&s)[4]) {
        float u = 0.0f;
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, s[b][i]);
        top = quads_max(top);
        if (__any(top * c > over)) {
            // (rows that need not be lifted stay as they are, whatever the others do)
            const bool first = over == -INFINITY;
            const float to = top * c > over ? m + top : m;
            const float up = to - m;
            const float f = first ? 1.0f : factor_of(-up * c);
            u = first ? kNever : up * c;
            if (top != -INFINITY) over = kLag;
            m = to;
            l *= f;
            if (!APART) rescale(f);
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[b][i] -= up;
        }
        float sum = 0.0f;  // of the tile first: beside a strong key's, one faint weight is nothing
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[b][i] = __builtin_amdgcn_exp2f(F32 ? s[b][i] * c : s[b][i]);
                sum += s[b][i];
            }
        l += sum;
        return u;
    }
    // Weights of 64 keys times their scales, relative to the row's own exponent, which
    // `most` lifts.  `hidden`: keys that the row does not see.
    __device__ __forceinline__ void weigh(f4_t (&s)[4], const float *scales, uint32_t hidden,
                                          float u) {
        float most = -kNever;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const f4_t t = *(const f4_t *)(scales + 16 * b);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[b][e] = hidden >> (4 * b + e) & 1 ? 0.0f : mantissa(s[b][e], t[e]);
                most = fmaxf(most, power(s[b][e], t[e]));
            }
        }
        rescale(lifted_to(ref, u, quads_max(most)));
        asm volatile("" ::: "memory");  // (the scales are read again, not held)
        const int down = kShift - own_exponent(ref);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const f4_t t = *(const f4_t *)(scales + 16 * b);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[b][e] = __builtin_amdgcn_ldexpf(s[b][e],
                                                  __builtin_amdgcn_frexp_expf(t[e]) + down);
        }
    }
    // The maximum in powers of two, minus infinity if there was none.
    __device__ __forceinline__ float top() const { return over == -INFINITY ? over : m * c; }
};

//
// One tile's room to a wave: K is requested again as soon as the scores are formed, V
// as soon as it is mixed, and the other waves cover what that leaves open.
// APART: every row has its own exponent.  Without, the loop ends early where scales lie too
// far apart for one (span.apart()): what it leaves is of no use then.  FOLD: sums of many
// tiles are put aside (which a wave of fewer than kFold + kFold / 2 never does).
template <int DIM, bool F32, bool ONCE, int NR, bool APART, bool FOLD>
__device__ __forceinline__ void step_loop(Block<DIM, F32> (&w)[NR], const StepFiller<DIM> &f,
                                          const Reach<kStepKeys> &r, int t, int t1, int stride,
                                          int top_lo, uint8_t *lds, int (&look)[4], Span8 &span,
                                          float k_factor) {
    using B = Block<DIM, F32>;
    constexpr int kAll = StepFiller<DIM>::kAll, kCodes = StepFiller<DIM>::kCodes;
    const int lane = f.lane, g = lane / 16;
    // lane i of 16 names the address of half a piece of the (i / 2)-th of its
    // eight keys and receives column i of all eight
    const int i2 = lane % 16 / 2;
    const int vkey = (i2 < 4 ? 4 * g + i2 : 12 + 4 * g + i2);
    const uint8_t *vrow = lds + kCodes + vkey * DIM + 8 * (lane % 2);
    float *ksc = (float *)(lds + 2 * kCodes);
    float *vsc = ksc + kStepKeys;
    int i = 0;  // the tile's lane in look
    Total<B> total[NR];
    bool aside = false;
    for (int count = 1; t < t1; t += stride, ++count) {
        const int k0 = r.key(t), next = r.key(t + stride);
        const bool more = t + stride < t1, masked = !r.all(k0, kStepKeys, top_lo);
        f4_t s[NR][4];
        Q4_WAIT_VMCNT(kAll);  // outstanding: K, then V
        asm volatile("" ::: "memory");
        const float k_mine = ksc[lane];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
#pragma unroll
            for (int n = 0; n < NR; ++n) s[n][b] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
            const int key = 16 * b + lane % 16;
#pragma unroll
            for (int j = 0; j < DIM / 64; ++j) {
                const u4_t x =
                    *(const u4_t *)(lds + key * DIM + (((4 * j + g) ^ swz8<DIM>(key)) * 16));
                const h8_t a0 = codes8(x[0], x[1]), a1 = codes8(x[2], x[3]);
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int y = 0; y < B::kParts; ++y) {
                        s[n][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, w[n].q[y][2 * j],
                                                                         s[n][b], 0, 0, 0);
                        s[n][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            a1, w[n].q[y][2 * j + 1], s[n][b], 0, 0, 0);
                    }
            }
        }
        // an infinite scale is no number either
        if (__builtin_expect(__any(fabsf(k_mine) == INFINITY), 0)) {
            if (fabsf(k_mine) == INFINITY) ksc[lane] = NAN;
            Q4_WAIT_LGKM0();
            asm volatile("" ::: "memory");
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            f4_t x = *(const f4_t *)(ksc + 16 * b + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!F32) x[e] *= k_factor;
#pragma unroll
                for (int n = 0; n < NR; ++n) s[n][b][e] = fmaf(s[n][b][e], x[e], -w[n].m);
            }
        }
        uint32_t hidden[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) hidden[n] = 0;
        if (masked) {
            asm volatile("; masked tile");  // a branch, not a select in every tile
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!w[n].sees(k0 + 16 * b + 4 * g + e, r.sinks)) {
                            s[n][b][e] = -INFINITY;
                            hidden[n] |= 1u << (4 * b + e);
                        }
        }
        Q4_WAIT_LGKM0();
        asm volatile("" ::: "memory");
        int page[4];
        if (more) {
            i = (i + 1) % 64;
            if (__builtin_expect(i == 0, 0)) {
                const int mine = r.key(min(t + stride + lane * stride, t1 - 1));
#pragma unroll
                for (int x = 0; x < 4; ++x) look[x] = f.look(mine + 16 * x);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) page[x] = __builtin_amdgcn_readlane(look[x], i);
            f.template fill<ONCE>(r, page, next, lds, false);
        }
        float u[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) u[n] = w[n].template soften<APART>(s[n]);
        // outstanding: V, then the next K
        if (more)
            Q4_WAIT_VMCNT(kAll);
        else
            Q4_WAIT_VMCNT(0);
        asm volatile("" ::: "memory");
        {
            const float t4 = vsc[lane];
            if (!APART) {
                // V's scales against the largest so far
                const int was = span.top;
                if (span.take(t4)) {
                    // (no way out of the loop here, which would cost registers: the next
                    // tile, whose keys are on their way, is the last)
                    if (__builtin_expect(span.apart(), 0)) t1 = min(t1, t + 2 * stride);
                    const float fall = __builtin_amdgcn_ldexpf(1.0f, was - span.top);
#pragma unroll
                    for (int n = 0; n < NR; ++n) w[n].rescale(fall);
                }
                vsc[lane] = relative(t4, span.top, B::kShift);
            } else {
                vsc[lane] = number(t4);
            }
        }
        Q4_WAIT_LGKM0();
        asm volatile("" ::: "memory");
        if (APART) {
#pragma unroll
            for (int n = 0; n < NR; ++n) w[n].weigh(s[n], vsc + 4 * g, hidden[n], u[n]);
        } else {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const f4_t x = *(const f4_t *)(vsc + 16 * b + 4 * g);
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][b][e] *= x[e];
            }
        }
        if (!APART && masked) {
            asm volatile("; masked tile");
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (hidden[n] >> (4 * b + e) & 1) s[n][b][e] = 0.0f;
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            h8_t p[NR][2];
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float y = s[n][2 * b + e / 4][e % 4];
                    const _Float16 hi = (_Float16)y;
                    p[n][0][e] = hi;
                    p[n][1][e] = (_Float16)(y - (float)hi);
                }
            // (two columns side by side: the two parts of one depend on each other)
#pragma unroll
            for (int d = 0; d < DIM / 16; d += 2) {
                h8_t a[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const i2_t x = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                        (lds_i2_t)(vrow + b * 32 * DIM + (((d + i) ^ swz8<DIM>(vkey)) * 16)));
                    a[i] = codes8((uint32_t)x[0], (uint32_t)x[1]);
                }
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int n = 0; n < NR; ++n)
                            w[n].o[d + i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                a[i], p[n][y], w[n].o[d + i], 0, 0, 0);
            }
        }
        Q4_WAIT_LGKM0();
        asm volatile("" ::: "memory");
        if (more) f.template fill<ONCE>(r, page, next, lds, true);
        if (FOLD && __builtin_expect(count % kFold == 0 && t1 - t > stride * (kFold / 2), 0)) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
                total[n].fold(w[n], APART ? own_exponent(w[n].ref) : span.top, aside);
            aside = true;
            // (none of these between the copies that are counted)
            Q4_WAIT_VMCNT(0);
            asm volatile("" ::: "memory");
        }
    }
    if (__builtin_expect(aside, 0))
#pragma unroll
        for (int n = 0; n < NR; ++n)
            total[n].back(w[n], APART ? own_exponent(w[n].ref) : span.top);
}

// Rows `first` to `last` (up to 16 NR) of the tile of rows row0 to row1, by W waves.  True
// if the scales of a wave's keys lie too far apart (without APART): nothing is written.
template <int DIM, bool F32, bool ONCE, int W, int NR, bool APART, bool FOLD>
__device__ __forceinline__ bool step_tile(const AttentionArgs &a, const Plan &pl, const Place &at,
                                          int hk, int split, int row0, int row1, int first,
                                          int last, uint8_t *lds, float (*ml)[W][kStepRows],
                                          uint32_t *votes, int wave) {
    constexpr int kPitch = DIM + 4, kShare = kStepRows * kPitch * 4;
    static_assert(2 * StepFiller<DIM>::kCodes + 2 * kStepKeys * 4 <= kShare && kShare % 256 == 0,
                  "a wave's tile, later its rows");
    const int position0 = at.kv - at.rows / pl.group;
    const int p0 = position(a, position0, row0 / pl.group);
    const int p1 = position(a, position0, (row1 - 1) / pl.group);
    const Reach<kStepKeys> r(a, p0, p1);
    const int top_lo = a.window && p1 >= a.window ? p1 - a.window + 1 : 0;
    const int per = max((r.tiles + pl.splits - 1) / pl.splits, pl.least);
    const int t0 = min(split * per, r.tiles);
    const int t1 = first < last ? min(t0 + per, r.tiles) : t0;
    // (two ways to name the lane: what the usual path has computed from it would else be
    // kept through its loop for the other)
    const int lane = APART ? __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u))
                           : threadIdx.x % 64;
    const int g = lane / 16;
    uint8_t *mine = lds + wave * kShare;
    const StepFiller<DIM> f(a, at.s, hk, lane);
    Block<DIM, F32> w[NR];
    const int t = t0 + wave;
    int look[4] = {-1, -1, -1, -1};
    {
        typename Block<DIM, F32>::Raw raw[NR];
        if (t < t1) {
            const int k = r.key(min(t + lane * W, t1 - 1));
#pragma unroll
            for (int x = 0; x < 4; ++x) look[x] = f.look(k + 16 * x);
        }
#pragma unroll
        for (int n = 0; n < NR; ++n)
            w[n].request(raw[n], a, at, pl.group, hk, first + 16 * n + lane % 16, position0,
                         g);
        if (t < t1) {
            int page[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) page[x] = __builtin_amdgcn_readlane(look[x], 0);
            f.template fill<ONCE>(r, page, r.key(t), mine, false);
            f.template fill<ONCE>(r, page, r.key(t), mine, true);
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) w[n].take(raw[n]);
#pragma unroll
        for (int n = 0; n < NR; ++n) w[n].clear();
    }
    Span8 span;
    step_loop<DIM, F32, ONCE, NR, APART, FOLD>(w, f, r, t, t1, W, top_lo, mine, look, span,
                                               finite(a.scale * kLog2e));
    if (!APART && __builtin_expect(span.apart(), 0)) {
        if (lane == 0) votes[wave] = 1;
        __syncthreads();
        return true;
    }
    // join the waves
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        w[n].l = quads_sum(w[n].l);
        w[n].m = w[n].top();
        if (g == 0) {
            ml[0][wave][16 * n + lane] = w[n].m;
            ml[1][wave][16 * n + lane] = w[n].l;
        }
    }
    if (!APART && lane == 0) votes[wave] = 0;
    __syncthreads();
    if (!APART) {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) any |= votes[i];
        if (__builtin_expect(uniform((int)any), 0)) return true;
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int rr = 16 * n + lane % 16;
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < W; ++i) m = fmaxf(m, ml[0][i][rr]);
        const float fs = factor_of(w[n].m - (m == -INFINITY ? 0.0f : m));
        if (rr < last - first) {
            const int top = APART ? own_exponent(w[n].ref) : span.top;
            float *row = (float *)mine + rr * kPitch + 4 * g;
#pragma unroll
            for (int d = 0; d < DIM / 16; ++d) {
                f4_t v;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = __builtin_amdgcn_ldexpf(w[n].o[d][e], top - w[n].kShift) * fs;
                *(f4_t *)(row + 16 * d) = v;
            }
        }
    }
    __syncthreads();
    for (int e = 64 * wave + lane; e < (last - first) * (DIM / 4); e += 64 * W) {
        const int rr = e / (DIM / 4), d = e % (DIM / 4) * 4;
        f4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
        float m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) m = fmaxf(m, ml[0][i][rr]);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const f4_t v = *(const f4_t *)((const float *)(lds + i * kShare) + rr * kPitch + d);
#pragma unroll
            for (int x = 0; x < 4; ++x) o[x] += v[x];
            l += ml[1][i][rr] * factor_of(ml[0][i][rr] - (m == -INFINITY ? 0.0f : m));
        }
        const int token = (first + rr) / pl.group;
        const int64_t out = (int64_t)(at.first + token) * a.q_heads + hk * pl.group +
                            (first + rr) % pl.group;
        if (pl.splits > 1 && d == 0) put_ml(a, pl, split, out, m, l);
        if (pl.splits > 1 && t0 >= t1) continue;
        put4<F32>(a, pl, split, out, DIM, d, o, l, position0 + token >= 0);
    }
    return false;
}

// Tile `w` of up to 64 conversations, the longest first: the first tiles of all, then
// what further ones there are.
__device__ __forceinline__ Place longest_first(const AttentionArgs &a, int group, int w) {
    const int lane = threadIdx.x % 64, s = min(lane, a.batch - 1);
    const bool held = lane < a.batch;
    const int b = min(max(a.q_start[s], 0), a.n), e = min(max(a.q_start[s + 1], b), a.n);
    const int kv = max(a.kv_len[s], 0);
    const int rows = (e - b) * group;
    int who, tile = 0;
    if (w < a.batch) {
        // (no two conversations have one key)
        const int key = (rows ? min(kv, (1 << 24) - 1) << 6 : 0) | lane;
        int before = 0;
        for (int i = 0; i < a.batch; ++i) before += __builtin_amdgcn_readlane(key, i) > key;
        who = __ffsll((unsigned long long)__ballot(held && before == w)) - 1;
    } else {
        const int more = held ? max((rows + kStepRows - 1) / kStepRows - 1, 0) : 0;
        int sum = more;
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) {
            const int x = __shfl_up(sum, i);
            if (lane >= i) sum += x;
        }
        const uint64_t past = __ballot(sum > w - a.batch);
        who = past ? __ffsll((unsigned long long)past) - 1 : 0;
        tile = past ? w - a.batch + 1 - __builtin_amdgcn_readlane(sum - more, who) : -1;
    }
    who = uniform(who);
    Place p;
    p.s = who;
    p.first = __builtin_amdgcn_readlane(b, who);
    p.rows = __builtin_amdgcn_readlane(rows, who);
    p.kv = __builtin_amdgcn_readlane(kv, who);
    p.tile = uniform(tile);
    return p;
}

// ONCE: a conversation's rows are one tile, most likely.
template <bool ONCE> __device__ __forceinline__ Place step_place(const Call &c) {
    const int w = c.base + (int)blockIdx.z;
    return ONCE && c.a.batch <= 64 ? longest_first(c.a, c.pl.group, w)
                                   : find_tile<kStepRows>(c.a, c.pl.group, w);
}

template <int DIM, bool F32, bool ONCE, int W, bool FOLD>
__global__ __launch_bounds__(64 * W, DIM > 128 ? 1 : 2) void step_kernel(Call c) {
    __shared__ __align__(1024) uint8_t lds[W * kStepRows * (DIM + 4) * 4];
    __shared__ float ml[2][W][kStepRows];
    __shared__ uint32_t votes[W];
    const int hk = blockIdx.x, split = blockIdx.y, wave = uniform(threadIdx.x / 64);
    {
        const Place at = step_place<ONCE>(c);
        const int row0 = at.tile * kStepRows;
        if (row0 < 0 || row0 >= at.rows) return;
        const int row1 = min(row0 + kStepRows, at.rows);
        const bool apart =
            row1 - row0 <= 16
                ? step_tile<DIM, F32, ONCE, W, 1, false, FOLD>(c.a, c.pl, at, hk, split, row0,
                                                               row1, row0, row1, lds, ml, votes,
                                                               wave)
                : step_tile<DIM, F32, ONCE, W, 2, false, FOLD>(c.a, c.pl, at, hk, split, row0,
                                                               row1, row0, row1, lds, ml, votes,
                                                               wave);
        if (!apart) return;
    }
    const Call &again = call_again();
    const Place at = step_place<ONCE>(again);
    const int row0 = at.tile * kStepRows, row1 = min(row0 + kStepRows, at.rows);
#pragma nounroll
    for (int first = row0; first < row1; first += 16) {
        __syncthreads();
        step_tile<DIM, F32, ONCE, W, 1, true, FOLD>(again.a, again.pl, at, hk, split, row0, row1,
                                                    first, min(first + 16, row1), lds, ml, votes,
                                                    wave);
    }
}

// ---- many rows: waves of 32 rows share each key tile ------------------------
// RW waves of 32 rows work on one key tile; KW such groups take every KW-th tile
// each and are joined through LDS at the end.  A tile is brought to binary16 once,
// on its way into LDS: its codes are loaded to registers a tile ahead, written to
// the other of two stages while this one is worked on, and read there by all RW
// waves.  Both products are v_mfma_f32_32x32x16_f16 on transposed scores; weights of
// float32 rows are held in two parts, those of binary16 rows rounded to one, as the
// result is: prompts of 2438 of 5001 and 3146 tokens are off by 2.9e-4 of their norm,
// with two parts by 2.1e-4 (the result's own rounding), but those take 403 us instead
// of 321, and full prompts of both lengths 491 instead of 384.
//
// Bound by vector instructions, 370 to 64 keys of 32 rows, of which 32 exponentials take
// four times as long; they hardly overlap with the matrix cores (busy for 33% of the
// cycles) at two waves to a SIMD, where waits for LDS and barriers take the rest;
// priorities change nothing (316 to 326 us).  What brought them down: codes converted
// once for all waves (they were half of the instructions when each wave converted its
// own), scores less the running maximum by one fused operation, no rescaling while the
// maximum lags by less than 2^8.  Eight waves on a key tile, which halves the
// conversions again, gained nothing (prompts of 5001 and 3146 tokens 406 us, four
// waves 390).
//
// Every wave brings 16 keys of K and V; wide float32 rows, whose registers are few,
// take half as many keys a tile, and a wave brings 16 of K or of V (44 prompts of 356
// tokens, 16 + 4 heads of 256: 343 us, with whole tiles 517).
template <int DIM, bool F32, int RW, int KW> struct Pass {
    static constexpr bool kBoth = !(DIM > 128 && F32 && RW > 2);
    static constexpr int KT = kBoth ? 16 * RW : 8 * RW;
    static constexpr int kTile = KT * DIM * 2;
    static constexpr int kPitch = DIM + 4, kShare = 32 * kPitch * 4;
    static constexpr int kStages = KW * 4 * kTile;
    static constexpr int kLds = RW * KW * kShare > kStages ? RW * KW * kShare : kStages;
    static constexpr int kThreads = 64 * RW * KW;
    static constexpr int kWavesPerSimd = DIM > 128 ? 1 : 2;
};

// Where 16-byte piece `piece` of a staged key row lies: eight lanes of a wave write the
// even pieces of one row, then the odd ones, and eight others those of the next row,
// so the rows' places differ in parity (or the halves of a 512-byte row's); both
// kinds of reads touch every bank once, as with swz().
template <int DIM> __device__ __forceinline__ int place(int key, int piece) {
    if (DIM == 64) return piece ^ ((((key >> 1) & 1) << 2) | (((key >> 2) ^ (key >> 1)) & 1) | ((key >> 2) & 2));
    const int low = DIM == 128 ? ((key >> 2) & 3) ^ (key & 1) : (key >> 2) & 3;
    return piece ^ (((key & 3) << 2) | low) ^ (DIM == 256 ? (piece >> 4) & 1 : 0);
}

// Scales of a stage: of K, of V (against 2^top), and top.
template <int KT> struct alignas(16) Scales {
    float k[KT], v[KT];
    int top;
};

// One wave's 32 rows, as a Block's.
template <int DIM, bool F32> struct Rows {
    static constexpr int kParts = F32 ? 2 : 1;
    // weights as 2^kShift of the largest, which may lag behind by kLag (powers of two)
    static constexpr float kLag = F32 ? 1.0f : 8.0f;
    static constexpr int kShift = F32 ? 14 : 7;
    h8_t q[kParts][DIM / 16];
    f16x_t o[DIM / 32];
    float m, l, c, over;
    int p, lo;

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
        c = F32 ? finite(a.scale * kLog2e) : 1.0f;
        const int64_t at = (int64_t)(pl.first + token) * a.q_stride +
                           (int64_t)(hk * group + rr % group) * DIM + 8 * half;
        const u4_t *src = (const u4_t *)((const uint8_t *)a.q + at * (F32 ? 4 : 2));
#pragma unroll
        for (int s = 0; s < DIM / 16; ++s)
#pragma unroll
            for (int x = 0; x < kParts; ++x) raw.x[s * kParts + x] = src[s * (F32 ? 4 : 2) + x];
        m = 0.0f;
        over = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
    }
    __device__ __forceinline__ void take(const Raw &raw) {
        int e = 0;
        if (F32) {
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
    static constexpr int kQuads = DIM / 8;  // of o
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
    }
    __device__ __forceinline__ f4_t quad(int i) const {
        const f16x_t &x = o[i / 4];
        const int k = i % 4 * 4;
        return f4_t{x[k], x[k + 1], x[k + 2], x[k + 3]};
    }
    __device__ __forceinline__ void add(int i, f4_t x, float f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i / 4][i % 4 * 4 + e] = fmaf(x[e], f, o[i / 4][i % 4 * 4 + e]);
    }
    __device__ __forceinline__ void rescale(float f) {
#pragma unroll
        for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] *= f;
    }
    __device__ __forceinline__ float top() const { return over == -INFINITY ? over : m * c; }
    // One tile: binary16 codes of K and V in LDS, and its scales.
    template <int KT>
    __device__ __forceinline__ void step(const uint8_t *kbuf, const uint8_t *vbuf,
                                         const Scales<KT> &sc, int k0, bool masked, int sinks) {
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
                const h8_t k = *(const h8_t *)(row + place<DIM>(key, 2 * d + half) * 16);
#pragma unroll
                for (int x = 0; x < kParts; ++x)
                    s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[x][d], s[t], 0, 0, 0);
            }
        }
#pragma unroll
        for (int t = 0; t < KT / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const f4_t x = *(const f4_t *)(sc.k + t * 32 + 2 * i + 4 * half);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[t][i + e] = fmaf(s[t][i + e], x[e], -m);
            }
        uint32_t hidden = 0;
        if (masked) {
            asm volatile("; masked tile");
#pragma unroll
            for (int t = 0; t < KT / 32; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!sees(k0 + t * 32 + 8 * (i / 4) + 4 * half + i % 4, sinks)) {
                        s[t][i] = -INFINITY;
                        hidden |= 1u << (16 * t + i);
                    }
        }
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < KT / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
        top = halves_max(top);
        if (__any(top * c > over)) {
            // (rows that need not be lifted stay as they are, whatever the others do)
            const bool first = over == -INFINITY;
            const float to = top * c > over ? m + top : m;
            const float up = to - m;
            const float f = first ? 1.0f : factor_of(-up * c);
            if (top != -INFINITY) over = kLag;
            m = to;
            l *= f;
            rescale(f);
#pragma unroll
            for (int t = 0; t < KT / 32; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[t][i] -= up;
        }
        h8_t w[KT / 16][kParts];
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < KT / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const f4_t x = *(const f4_t *)(sc.v + t * 32 + 2 * i + 4 * half);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float y = __builtin_amdgcn_exp2f(F32 ? s[t][i + e] * c : s[t][i + e]);
                    sum += y;
                    s[t][i + e] = y * x[e];
                }
            }
        l += sum;
        if (masked) {
            asm volatile("; masked tile");
#pragma unroll
            for (int t = 0; t < KT / 32; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (hidden >> (16 * t + i) & 1) s[t][i] = 0.0f;
        }
#pragma unroll
        for (int b = 0; b < KT / 16; ++b)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = s[b / 2][8 * (b % 2) + i];
                const _Float16 hi = (_Float16)y;
                w[b][0][i] = hi;
                if (F32) w[b][kParts - 1][i] = (_Float16)(y - (float)hi);
            }
#pragma unroll
        for (int b = 0; b < KT / 16; ++b) {
            const int key = 16 * b + 4 * half + lane % 16 / 4;
            const int piece = 2 * (lane / 16 % 2) + lane % 4 / 2;
            const uint8_t *r0 = vbuf + key * DIM * 2 + 8 * (lane % 2);
            const uint8_t *r1 = r0 + 8 * DIM * 2;
#pragma unroll
            for (int d = 0; d < DIM / 32; ++d) {
                const s4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s4_t)(r0 + place<DIM>(key, 4 * d + piece) * 16));
                const s4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s4_t)(r1 + place<DIM>(key + 8, 4 * d + piece) * 16));
                const h8_t v = __builtin_bit_cast(
                    h8_t, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                for (int x = 0; x < kParts; ++x)
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, w[b][x], o[d], 0, 0, 0);
            }
        }
    }
};

// This workgroup's tile of R rows, those with the most keys first; false if it has none.
template <int R> __device__ __forceinline__ bool pass_place(const Call &c, Place &at) {
    at = find_tile<R>(c.a, c.pl.group, c.base + (int)blockIdx.z);
    const int count = (at.rows + R - 1) / R;
    if (at.tile < 0 || at.tile >= count) return false;
    at.tile = count - 1 - at.tile;
    return true;
}

template <int DIM, bool F32, int RW, int KW>
__global__ __launch_bounds__((Pass<DIM, F32, RW, KW>::kThreads),
                             (Pass<DIM, F32, RW, KW>::kWavesPerSimd)) void pass_kernel(Call c) {
    const AttentionArgs &a = c.a;
    const Plan &pl = c.pl;
    using P = Pass<DIM, F32, RW, KW>;
    using W = Rows<DIM, F32>;
    constexpr bool kBoth = P::kBoth;
    constexpr int KT = P::KT, kTile = P::kTile, R = 32 * RW, kLoads = DIM / 64;
    __shared__ __align__(1024) uint8_t lds[P::kLds];
    __shared__ Scales<KT> scales[2][KW];
    __shared__ float ml[2][KW][R];
    __shared__ uint32_t votes[KW];
    const int hk = blockIdx.x;
    Place at;
    if (!pass_place<R>(c, at)) return;
    const int position0 = at.kv - at.rows / pl.group;
    const int row0 = at.tile * R, row1 = min(row0 + R, at.rows);
    const int p0 = position(a, position0, row0 / pl.group);
    const int p1 = position(a, position0, (row1 - 1) / pl.group);
    const Reach<KT> r(a, p0, p1);
    const int top_lo = a.window && p1 >= a.window ? p1 - a.window + 1 : 0;
    const int lane = threadIdx.x % 64, half = lane / 32, wave = uniform(threadIdx.x / 64);
    const int rw = wave % RW, kw = wave / RW;
    const int mine = rw * 32 + lane % 32, row = row0 + mine;
    W w;
    {
        typename W::Raw raw;
        w.request(raw, a, at, pl.group, hk, row, position0);
        w.take(raw);
    }
    int top = kNoExponent;  // of the values in o
    const int tiles = max((r.tiles - kw + KW - 1) / KW, 0);  // this group's
    const int rounds = uniform((r.tiles + KW - 1) / KW);     // the first group's
    const Source f(a, at.s, hk);
    uint8_t *stages = lds + kw * 4 * kTile;
    const auto key_of = [&](int i) { return r.key(kw + i * KW); };
    // a tile's loads: this wave's 16 rows of K and V (or of one of them, in kx), and the
    // scales of V (first wave) or K (second), a key to a lane
    const int group = rw % (KT / 16);
    u4_t kx[kLoads], vx[kLoads];
    float sx = 0.0f;
    const auto look = [&](int i) { return f.look(key_of(min(i, tiles - 1)) + lane % KT); };
    const auto load = [&](int i, int pages) {
        const int k0 = key_of(i), k = k0 + 16 * group;
        const int64_t at16 =
            f.row(__builtin_amdgcn_readlane(pages, 16 * group), k) * DIM + lane * 16;
        const uint8_t *src = kBoth || rw < KT / 16 ? f.k : f.v;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            kx[j] = *(const u4_t *)(src + at16 + j * 1024);
            if (kBoth) vx[j] = *(const u4_t *)(f.v + at16 + j * 1024);
        }
        if (rw < 2) sx = *(const float *)f.scale(r, pages, k0 + lane % KT, rw == 0);
    };
    const float k_factor = F32 ? 1.0f : finite(a.scale * kLog2e);
    Span8 span;  // of the wave that stages V's scales
    const auto stage = [&](int i) {
        uint8_t *dst = stages + (i & 1) * 2 * kTile + (kBoth || rw < KT / 16 ? 0 : kTile);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int key = 16 * group + j * (1024 / DIM) + lane / (DIM / 16);
            const int piece = lane % (DIM / 16) * 2;
            uint8_t *even = dst + key * DIM * 2 + place<DIM>(key, piece) * 16;
            uint8_t *odd = dst + key * DIM * 2 + place<DIM>(key, piece + 1) * 16;
            *(h8_t *)even = codes8(kx[j][0], kx[j][1]);
            *(h8_t *)odd = codes8(kx[j][2], kx[j][3]);
            if (!kBoth) continue;
            *(h8_t *)(even + kTile) = codes8(vx[j][0], vx[j][1]);
            *(h8_t *)(odd + kTile) = codes8(vx[j][2], vx[j][3]);
        }
        Scales<KT> &sc = scales[i & 1][kw];
        if (rw == 0) {
            span.take(sx);
            if (lane < KT) sc.v[lane] = relative(sx, span.top, W::kShift);
            if (lane == 0) sc.top = span.top;
        } else if (rw == 1 && lane < KT) {
            sc.k[lane] = fabsf(sx) <= FLT_MAX ? sx * k_factor : NAN;
        }
    };
    Total<W> total;
    int pages = -1;
    if (tiles > 0) {
        load(0, look(0));
        pages = look(1);
        stage(0);
        if (tiles > 1) load(1, pages);
        pages = look(2);
    }
    for (int i = 0; i < rounds; ++i) {
        __syncthreads();
        if (i + 1 < tiles) {
            stage(i + 1);
            if (i + 2 < tiles) {
                load(i + 2, pages);
                pages = look(i + 3);
            }
        }
        if (i >= tiles) continue;
        __builtin_amdgcn_sched_barrier(0);
        const Scales<KT> &sc = scales[i & 1][kw];
        const int now = uniform(sc.top);
        if (now != top) {
            w.rescale(__builtin_amdgcn_ldexpf(1.0f, top - now));
            top = now;
        }
        const int k0 = key_of(i);
        const uint8_t *kbuf = stages + (i & 1) * 2 * kTile;
        w.template step<KT>(kbuf, kbuf + kTile, sc, k0, !r.all(k0, KT, top_lo), r.sinks);
        if (i % kFold == kFold - 1 && tiles - i > kFold / 2) total.fold(w, top, i >= kFold);
    }
    // Scales too far apart for one exponent are asked for at the end alone (as soon as
    // they are met, in the loop: attend both prompts in 329 us, so in 322).
    if (rw == 0 && lane == 0) votes[kw] = span.apart();
    __syncthreads();
    uint32_t apart = 0;
#pragma unroll
    for (int i = 0; i < KW; ++i) apart |= votes[i];
    if (__builtin_expect(uniform((int)apart), 0)) {
        // 16 rows to a wave, which takes all keys
        constexpr int kAll = RW * KW;
        const Call &again = call_again();
        Place at;
        pass_place<R>(again, at);
        const int row0 = at.tile * R, row1 = min(row0 + R, at.rows);
#pragma nounroll
        for (int x = 0; x < R / 16; x += kAll) {
            const int first = row0 + 16 * (x + wave);
            __syncthreads();
            step_tile<DIM, F32, false, 1, 1, true, true>(
                again.a, again.pl, at, blockIdx.x, 0, row0, row1, min(first, row1),
                min(first + 16, row1), lds + wave * P::kShare,
                (float(*)[1][kStepRows])(&ml[0][0][0] + wave * 2 * kStepRows), nullptr, 0);
        }
        return;
    }
    if (tiles >= kFold + kFold / 2) total.back(w, top);
    // the values' own magnitude again, the maximum in powers of two
#pragma unroll
    for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            w.o[d][i] = __builtin_amdgcn_ldexpf(w.o[d][i], top - W::kShift);
    float l = halves_sum(w.l);
    const float m = w.top();
    if (KW > 1) {
        // join the groups: the first takes over its rows' sum
        if (lane < 32) ml[0][kw][mine] = m, ml[1][kw][mine] = l;
        __syncthreads();
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < KW; ++i) most = fmaxf(most, ml[0][i][mine]);
        const float zero = most == -INFINITY ? 0.0f : most;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < KW; ++i) l += ml[1][i][mine] * factor_of(ml[0][i][mine] - zero);
        const float fs = factor_of(m - zero);
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
        if (wave < RW && lane < 32) ml[1][0][mine] = l;
        __syncthreads();
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
            put_y4<F32>(a, out, DIM, d, o, ml[1][0][rr], position0 + token >= 0);
        }
        return;
    }
    if (row >= row1) return;
    const int64_t out = (int64_t)(at.first + row / pl.group) * a.q_heads + hk * pl.group +
                        row % pl.group;
#pragma unroll
    for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            put_y4<F32>(a, out, DIM, 32 * d + 2 * i + 4 * half,
                        f4_t{w.o[d][i], w.o[d][i + 1], w.o[d][i + 2], w.o[d][i + 3]}, l,
                        w.p >= 0);
}

// ---- joining the parts of many rows -----------------------------------------
// A wave to a row, where there are rows enough to fill the device that way: the
// parts' maxima and sums in its lanes, then the rows' elements, four to a lane, the
// parts dealt to the lanes that a row leaves free.
template <int DIM, bool F32>
__global__ __launch_bounds__(256) void join_rows_kernel(AttentionArgs a, Plan pl) {
    constexpr int kCols = DIM / 4, kGroups = 64 / kCols;
    const int lane = threadIdx.x % 64;
    const int64_t rows = (int64_t)a.n * a.q_heads;
    const int64_t row = uniform((int)(blockIdx.x * 4 + threadIdx.x / 64));
    if (row >= rows) return;
    const int token = (int)(row / a.q_heads);
    float m = -INFINITY, l = 0.0f;
    if (lane < pl.splits) {
        const float *ml = pl.part_ml + (lane * rows + row) * 2;
        m = ml[0], l = ml[1];
    }
    constexpr int kAhead = 4;
    f4_t ahead[kAhead];
    const float *src = pl.part + row * DIM + lane % kCols * 4;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int part = lane / kCols + i * kGroups;
        if (part < pl.splits) ahead[i] = *(const f4_t *)(src + part * rows * DIM);
    }
    const int s = find_last(a.batch, [&](int i) { return a.q_start[i] <= token; });
    const meta_t qs = meta(a.q_start);
    const int begin = min(max(qs[s], 0), a.n), end = min(max(qs[s + 1], begin), a.n);
    if (token < begin || token >= end) return;
    const bool sees = max(meta(a.kv_len)[s], 0) - end + token >= 0;
    float top = m;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) top = fmaxf(top, __shfl_xor(top, i));
    // a part that saw none of the row's keys wrote no elements: marked by -1
    const bool used = m != -INFINITY || l != 0.0f;
    const float f = used ? factor_of(m - (top == -INFINITY ? 0.0f : top)) : -1.0f;
    l = used ? l * f : 0.0f;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) l += __shfl_xor(l, i);
    f4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
    const int rounds = (pl.splits + kGroups - 1) / kGroups;
    for (int i = 0; i < rounds; ++i) {
        const int part = lane / kCols + i * kGroups;
        const float g = __shfl(f, min(part, 63));
        if (part >= pl.splits || g == -1.0f) continue;
        f4_t v;
        if (i == 0)
            v = ahead[0];
        else if (i == 1)
            v = ahead[1];
        else if (i == 2)
            v = ahead[2];
        else if (i == 3)
            v = ahead[3];
        else
            v = *(const f4_t *)(src + part * rows * DIM);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += v[e] * g;
    }
#pragma unroll
    for (int i = kCols; i < 64; i <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], i);
    if (lane < kCols) put_y4<F32>(a, row, DIM, 4 * lane, o, l, sees);
}

// ---- choices on the host ----------------------------------------------------
struct Choice {
    int rows;   // of a tile: 32 (every wave on its own keys), 64 or 128 (waves share them)
    int waves;  // of a 32-row workgroup
    bool once;  // a conversation's rows are one such tile, likely
    int64_t tiles;
    int splits;
    int least;  // key tiles of a part, at least
    bool fold;  // a wave may take so many key tiles that their sums are put aside
    size_t part, bytes;  // workspace: bytes of the partial rows, and in all
};

// How a call is cut into work items.  The host knows the sizes, not the
// conversations' lengths: those may change between replays of a graph.
Choice choose(const AttentionArgs &a) {
    Choice ch;
    const int dim = a.cache.dim, heads = a.cache.heads;
    const int64_t rows = (int64_t)a.n * (a.q_heads / heads);
    const int64_t cus = device_shape().cus;
    // 32-row tiles where one holds a conversation's rows: it reads each key once.
    // With more rows 128-row tiles, if that gives every compute unit one.  Between
    // them 32-row tiles again, as long as one and a half times as many as there are
    // compute units do (two run on each at once): the conversation's tiles read its
    // keys side by side, from L2.  Else 64-row tiles, whose waves share them.  32- and
    // 64-row tiles (us; 32 + 8 heads of 128, binary16): 16 conversations of 8192 keys, 16
    // new tokens each, 107 and 160; one of 131072, 32 new tokens, 162 and 242; 256 new
    // tokens of 4112 51 and 67; 512 of 4112 80 and 67, 512 of 512 17.4 and 16.1.  The
    // rule takes a few short calls from the wrong side: 64 of 4112 25.8 and 21.6, four
    // times 32 of 2048 (heads of 64) 21.8 and 17.1.
    const bool one = rows <= (int64_t)kStepRows * a.batch;
    const bool few = 2 * (rows / 32 + a.batch) * heads <= 3 * cus;
    if (!one && (rows / 128 + (a.batch + 1) / 2) * heads >= cus)
        ch.rows = 128;
    else
        ch.rows = one || few ? 32 : 64;
    ch.once = one;
    ch.tiles = rows / ch.rows + a.batch;
    ch.waves = dim > 128 ? 2 : 4;
    ch.splits = ch.least = 1;
    ch.part = ch.bytes = 0;
    ch.fold = true;
    if (ch.rows > 32) return ch;  // (such tiles fill three quarters of the device, or all)
    // the items that are likely to have work: not all tiles do
    const int64_t likely = (rows / 32 > a.batch ? rows / 32 : a.batch) * heads;
    // the key tiles a row tile can have at most
    int64_t keys = (int64_t)a.table_stride << a.cache.page_shift;
    if (a.window) {
        const int64_t near = (int64_t)a.window + a.sinks + 2 * kStepRows + 2 * kStepKeys;
        if (near < keys) keys = near;
    }
    const int64_t most = (keys + kStepKeys - 1) / kStepKeys;
    // One conversation of many keys: half as many parts of twice the waves (4 + 1 heads and
    // 32 + 8 of 128: 20000 keys 13.3 us and 14.5, otherwise 14.0 and 17.8; 12000 keys
    // 12.6 and 13.1, otherwise 11.0 and 13.6; 131072 keys of 32 + 8 53.1 and 51.6, of
    // 16 + 4 heads of 256 60.9 and 55.2).
    const bool solo = ch.once && a.batch == 1 && most >= 256;
    if (solo) ch.waves *= 2;
    // workgroups that run at once: two to a compute unit, four of 64-wide heads
    const int64_t slots = cus * (dim > 64 ? 2 : 4) / (solo ? 2 : 1);
    // As many parts as run at once, of 1024 keys at least, or of what gives every slot
    // one where that is less; none where the conversations alone fill the device.
    // Four times as many, so that long conversations do not end alone, gain less
    // than writing and joining parts costs: 128 conversations of 100 to 2048
    // keys, one token each, 63 us so and 78 us, four tokens each 69 and 91; 16
    // of 8192, eight tokens of 64 heads each, 95 and 116.  Parts of 512, 1024 and
    // 2048 keys at least: 48 conversations of 200 to 4096 keys 53, 56 and 62; 24
    // of 800 to 16384 99, 99 and 101; others alike.
    int64_t splits = (slots + (a.batch == 1 ? 0 : likely - 1)) / likely;
    const int64_t fair = (most * likely + slots - 1) / slots;
    ch.least = fair > 16 ? 16 : fair < ch.waves ? ch.waves : (int)fair;
    // Up to 64 conversations come the longest first.  With more of them than fill the
    // device when each workgroup has eight waves (four), that evens out several
    // lengths better than parts do: 64 of 400 to 8192 keys 99 and 112 us, one to five
    // tokens each 120 and 131, 48 of 200 to 4096 45 and 54; short ones and equal ones
    // lose (64 of 25 to 512 keys 22 and 16, all of 4096 98 and 92).
    if (ch.once && a.batch <= 64 && 4 * likely > 5 * cus && most >= 32)
        splits = 1, ch.waves *= 2;
    // Few keys: the workgroup's own waves take them, eight (four), while there are
    // units to spare; and where half of them are busy anyhow (20 conversations of 50
    // to 1024 keys 13.7 us, in parts 16.5; eight of them 13.1 and 10.8).
    else if (!solo && ch.once && likely <= cus && (most / ch.least < 2 || (2 * likely > cus && most <= 16)))
        splits = 1, ch.waves *= 2;
    // (a part of the fewest keys, a tile to a wave, is not made longer by the rest: 700
    // keys in three parts, 10.2 us, in two 12.7; 4000 keys 10.4 and 12.3)
    const int64_t fit = (most + (ch.least > ch.waves ? 0 : ch.least - 1)) / ch.least;
    if (splits > fit) splits = fit;
    if (splits > kMaxSplits) splits = kMaxSplits;
    const int64_t out = (int64_t)a.n * a.q_heads;
    const int64_t room = (int64_t)kWorkspaceBytes / (out * (dim + 2) * 4);
    if (splits > room) splits = room;
    ch.splits = splits < 2 ? 1 : (int)splits;
    if (ch.splits == 1) ch.least = 1;
    // Without that code one conversation of 448 keys takes 9.3 us, with it 9.6; 32 of 400 to
    // 8192 with heads of 256 152 and 155.
    const int64_t per = (most + ch.splits - 1) / ch.splits;
    ch.fold = ((per > ch.least ? per : ch.least) + ch.waves - 1) / ch.waves >= kFold + kFold / 2;
    ch.part = ch.splits > 1 ? (size_t)ch.splits * (size_t)out * (size_t)dim * 4u : 0;
    ch.bytes = ch.splits > 1 ? ch.part + (size_t)ch.splits * (size_t)out * 8u : 0;
    return ch;
}

template <int DIM, bool F32, bool ONCE, int W>
void launch_step(const Call &c, const dim3 &grid, bool fold, hipStream_t stream) {
    if (fold)
        hipLaunchKernelGGL((step_kernel<DIM, F32, ONCE, W, true>), grid, dim3(64 * W), 0, stream, c);
    else
        hipLaunchKernelGGL((step_kernel<DIM, F32, ONCE, W, false>), grid, dim3(64 * W), 0, stream,
                           c);
}

template <int DIM, bool F32>
hipError_t run(const AttentionArgs &a, const Choice &ch, const Plan &pl, hipStream_t stream) {
    constexpr int W = DIM > 128 ? 2 : 4;
    // heads fastest: the tiles of one head of a conversation come to the same
    // die, eight heads to eight dies, and share its L2
    for (int64_t base = 0; base < ch.tiles; base += 65535) {
        const int64_t tiles = ch.tiles - base < 65535 ? ch.tiles - base : 65535;
        const dim3 grid((uint32_t)a.cache.heads, (uint32_t)ch.splits, (uint32_t)tiles);
        const Call c = {a, pl, (int)base};
        if (ch.rows == 128)
            hipLaunchKernelGGL((pass_kernel<DIM, F32, 4, 1>), grid, dim3(256), 0, stream, c);
        else if (ch.rows == 64)
            hipLaunchKernelGGL((pass_kernel<DIM, F32, 2, W>), grid, dim3(128 * W), 0, stream, c);
        else if (!ch.once)
            launch_step<DIM, F32, false, W>(c, grid, ch.fold, stream);
        else if (ch.waves == W)
            launch_step<DIM, F32, true, W>(c, grid, ch.fold, stream);
        else
            launch_step<DIM, F32, true, 2 * W>(c, grid, ch.fold, stream);
    }
    const int64_t out = (int64_t)a.n * a.q_heads;
    // Parts of many rows are joined a wave to a row, of few by a workgroup each (whole
    // calls, us): 8192 rows 101 and 104, the same of 256 new tokens of 4112 keys 51 and
    // 60, 1024 rows 25.7 and 29.1; 256 rows 66 and 63.
    if (ch.splits > 1 && ch.splits <= 64 && out >= 4 * device_shape().cus)
        hipLaunchKernelGGL((join_rows_kernel<DIM, F32>), dim3((uint32_t)((out + 3) / 4)), dim3(256),
                           0, stream, a, pl);
    else if (ch.splits > 1)
        hipLaunchKernelGGL((join_kernel<F32>), dim3((uint32_t)out), dim3(256), 0, stream, a, pl);
    return hipGetLastError();
}

template <bool F32>
hipError_t by_dim(const AttentionArgs &a, const Choice &ch, const Plan &pl, hipStream_t stream) {
    if (a.cache.dim == 64) return run<64, F32>(a, ch, pl, stream);
    if (a.cache.dim == 128) return run<128, F32>(a, ch, pl, stream);
    return run<256, F32>(a, ch, pl, stream);
}

}  // namespace

size_t attention8_workspace_bytes(const AttentionArgs &a) { return choose(a).bytes; }

int attention8_tile_rows(const AttentionArgs &a) { return choose(a).rows; }

hipError_t launch_attention8(const AttentionArgs &a, int x_f16, void *ws, hipStream_t stream) {
    const Choice ch = choose(a);
    const Plan pl = {a.q_heads / a.cache.heads, ch.splits, ch.least, (float *)ws,
                     (float *)((uint8_t *)ws + ch.part)};
    return x_f16 ? by_dim<false>(a, ch, pl, stream) : by_dim<true>(a, ch, pl, stream);
}

}  // namespace q4
