// Verification of drafted tokens against the target's probabilities.
//
// With p = softmax(l / T) of a row and q = softmax(g / T) of the draft's (all of q on
// the draft where there is none), draft d is taken iff u q(d) < p(d).  After the
// first one refused the next token is drawn from max(p - q, 0), after the last one
// from p: the lowest token whose cumulative weight passes u' times the total.
//
// A draw is a border among up to 10^5 shares, so weights and sums are 64-bit: the
// same token comes out whatever the order of the sums.  A weight 2^x is a table's
// entry (256 of them) times a polynomial of the third degree, off by 2e-13; weights
// below 2^-980 of a row's largest count as none, in every kernel by the same comparison,
// so that a part has a share exactly if a token in it has a weight.
//
// stats: every part of every row, one read: its largest logit and the sum of its
// weights (without draft logits both of all but the judged draft, so that taking it
// out costs no digits).  judge: each conversation's first refused draft.  rest (with
// draft logits): sums of max(p - q, 0) over the parts of that row.  pick: the part
// that the number falls into, then the token.  Few parts: rest judges, three launches.
// Without draft logits pick judges, and two are all.
//
// Measured: one conversation of four picked drafts over 151936 tokens 8.3 us, a chain of
// two launches; 12 conversations of up to three drafts over 32003 tokens 14 us, a
// chain of three; 64 conversations of up to six drafts over 151936 tokens (318 MB that
// stats has to read) 80 us, of which stats 61: ten operations of 64 bits and five
// others an element, 70% of its time, where the bytes alone are 44 us.
#include <float.h>

#include "q4_0_device.h"
#include "q4_0_internal.h"

namespace q4 {

namespace {

typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
typedef f4_t f4_any_t __attribute__((aligned(4)));
typedef h4_t h4_any_t __attribute__((aligned(2)));

constexpr int kPart = 2048;        // tokens of a part: one wave's, or four's
constexpr int kLoads = kPart / 256;
constexpr int kThreads = 256;      // of stats: four parts, or one
constexpr int kWaves = kThreads / 64;
constexpr int kPickThreads = 512;  // of the others: one part, or eight rows judged at once
constexpr int kPickWaves = kPickThreads / 64;
constexpr int kHeld = 2;           // parts that a lane keeps: rows of 262144 tokens need no more

// A part of a row: its largest logit, the sum of its weights relative to that
// logit (without draft logits the judged draft is in neither), and `at`: of a greedy
// row the first token that has the largest, else (as bits) the judged draft's logit,
// where it is in this part.  A sum that is no number: the part holds a logit that is
// NaN or plus infinity.
struct Stat {
    double sum;
    float top;
    int32_t at;
};

// How the next token is found.
enum { kNone, kGreedy, kPlain, kWithout, kRest };
// A conversation's judgement: the row that ends it and what follows, its largest
// logits and the reciprocals of its total weights (of p, of q), the number to draw
// with, its first best token.
struct Verdict {
    double p_share, q_share;
    float p_top, q_top, u;
    int row, how, draft, at;
};

// 2^(i / 256), computed by the compiler: square roots by Newton's method, and each
// entry a product of at most eight of them.
struct Table {
    double v[256];
    constexpr Table() : v() {
        double roots[8] = {};  // 2^(1/2), 2^(1/4), ..
        double of = 2.0;
        for (int k = 0; k < 8; ++k) {
            double x = of;
            for (int n = 0; n < 12; ++n) x = 0.5 * (x + of / x);
            roots[k] = of = x;
        }
        for (int i = 0; i < 256; ++i) {
            v[i] = 1.0;
            for (int k = 0; k < 8; ++k)
                if (i >> (7 - k) & 1) v[i] *= roots[k];
        }
    }
};
static __device__ const Table kTable = Table();

__device__ __forceinline__ void fill_table(double *table) {
    if (threadIdx.x < 256) table[threadIdx.x] = kTable.v[threadIdx.x];
}

// Weights exp(d / T) of differences d <= 0, from the table in LDS.
struct Power {
    const double *table;
    double c, least;  // 256 log2(e) / T, and the difference that stands for all below
    double faint;     // differences below this one have no weight
    __device__ __forceinline__ Power(const double *t, double heat)
        : table(t), c(369.3299304675746 / heat), least(-1010.0 * 0.6931471805599453 * heat),
          faint(-980.0 * 0.6931471805599453 * heat) {}
    // Sum of the weights of N differences, side by side: a single one is a chain of
    // ten operations and an LDS read.  None is below about 2^-1010, so that the
    // exponent is a plain addition.
    template <int N> __device__ __forceinline__ void of(const double (&d)[N], double (&w)[N]) const {
        const double magic = 6755399441055744.0;  // 1.5 2^52: the sum's low bits are the integer
        double r[N], z[N];
        uint32_t k[N];
        uint64_t t[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const double x = fmax(d[i], least), y = fma(x, c, magic);
            r[i] = fma(x, c, -(y - magic));
            k[i] = (uint32_t)__builtin_bit_cast(uint64_t, y);
            t[i] = __builtin_bit_cast(uint64_t, table[k[i] & 255]);
        }
        // e^z, z = r ln(2) / 256, |z| < 0.00136
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = fma(3.3083026805413713e-09, r[i], 3.6655655969101062e-06);
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = fma(z[i], r[i], 0.0027076061740622863);
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = fma(z[i], r[i], 1.0);
#pragma unroll
        for (int i = 0; i < N; ++i)
            w[i] = z[i] * __builtin_bit_cast(
                              double, (uint64_t)((uint32_t)(t[i] >> 32) + ((k[i] & ~255u) << 12))
                                              << 32 |
                                          (uint32_t)t[i]);
    }
    // The same, 0 where there is none.
    template <int N>
    __device__ __forceinline__ void exact(const double (&d)[N], double (&w)[N]) const {
        of(d, w);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = d[i] >= faint ? w[i] : 0.0;
    }
    __device__ __forceinline__ double exact(double d) const {
        const double one[1] = {d};
        double w[1];
        exact(one, w);
        return w[0];
    }
};

// Four neighbouring logits of a row from element i on; minus infinity past its end.
template <bool F16> __device__ __forceinline__ f4_t load4(const void *row, int i, int vocab) {
    f4_t x;
    if (i + 4 <= vocab) {
        if (!F16) return *(const f4_any_t *)((const float *)row + i);
        const h4_t h = *(const h4_any_t *)((const _Float16 *)row + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = (float)h[e];
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[e] = i + e >= vocab ? -INFINITY
                                  : (F16 ? (float)((const _Float16 *)row)[i + e]
                                         : ((const float *)row)[i + e]);
    }
    return x;
}
template <bool F16> __device__ __forceinline__ float load1(const void *row, int i) {
    return F16 ? (float)((const _Float16 *)row)[i] : ((const float *)row)[i];
}
// A lane's logits of a part: runs of four, 256 tokens apart, N from the `from`-th on.
template <bool F16, int N>
__device__ __forceinline__ void load_part(f4_t (&l)[N], const void *row, int part, int vocab,
                                          int from = 0) {
    const int base = part * kPart + from * 256 + threadIdx.x % 64 * 4;
    if ((part + 1) * kPart <= vocab) {
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = load4<F16>(row, base + i * 256, INT32_MAX);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = load4<F16>(row, base + i * 256, vocab);
    }
}
template <bool F16>
__device__ __forceinline__ const void *row_of(const void *p, int64_t row, int64_t stride) {
    return (const uint8_t *)p + row * stride * (F16 ? 2 : 4);
}

// Sums over a wave by lane moves: no LDS in between.
template <int CTRL, int ROWS> __device__ __forceinline__ double moved(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF,
                                                              false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL,
                                                              ROWS, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// x of this lane and all before it.
__device__ __forceinline__ double up_to(double x) {
    x += moved<0x111, 0xF>(x);  // one lane on within 16, two, four, eight
    x += moved<0x112, 0xF>(x);
    x += moved<0x114, 0xF>(x);
    x += moved<0x118, 0xF>(x);
    x += moved<0x142, 0xA>(x);  // the last of 16 to the next 16, of 32 to the next 32
    x += moved<0x143, 0xC>(x);
    return x;
}
__device__ __forceinline__ double lane_of(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double x) { return lane_of(up_to(x), 63); }

// The larger number; NaN if either is.
__device__ __forceinline__ float larger(float x, float y) {
    return __builtin_elementwise_maximum(x, y);
}
template <int CTRL> __device__ __forceinline__ float turned(float x) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float wave_max(float x) {
    x = larger(x, turned<0x121>(x));
    x = larger(x, turned<0x122>(x));
    x = larger(x, turned<0x124>(x));
    x = larger(x, turned<0x128>(x));
    uint32_t u = __builtin_bit_cast(uint32_t, x);
    auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    x = larger(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
    u = __builtin_bit_cast(uint32_t, x);
    r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return larger(__builtin_bit_cast(float, (uint32_t)r[0]),
                  __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) x = min(x, __shfl_xor(x, i));
    return x;
}

// The conversation that holds a row, if one does: its rows are [first, last].
struct Span {
    int s, first, last;
};
__device__ __forceinline__ bool span_of(const VerifyArgs &a, int s, Span &sp) {
    sp.s = s;
    sp.first = min(max(a.q_start[s], 0), a.n);
    sp.last = min(max(a.q_start[s + 1], sp.first), a.n) - 1;
    return sp.last >= sp.first;
}
// The last s with q_start[s] <= row, by all lanes of a wave.
__device__ __forceinline__ int holder(const VerifyArgs &a, int row) {
    const int lane = threadIdx.x % 64;
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64;
        const int i = lo + lane * step;
        const int last = __popcll(__ballot(i < hi && a.q_start[i] <= row)) - 1;
        lo += (last < 0 ? 0 : last) * step;
        hi = min(lo + step, hi);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}
__device__ __forceinline__ float heat_of(const VerifyArgs &a, int s) {
    return a.heat ? a.heat[s] : 1.0f;
}

// ---- every part of every row ------------------------------------------------
// A part to W waves of a workgroup, four where there are few: the chain is as short as
// it gets.  A row of logits is requested before the conversation that holds it is
// known, the draft's only then: those that judge nothing (each conversation's last, all
// of a greedy one) need not be there.
template <bool F16, int W>
__global__ __launch_bounds__(kThreads, 8) void stats_kernel(VerifyArgs a, Stat *stats, int parts) {
    constexpr int kParts = kWaves / W, kMine = kLoads / W;
    __shared__ double table[256];
    __shared__ double sums[W];
    __shared__ float tops[W];
    __shared__ int firsts[W];
    const int groups = (parts + kParts - 1) / kParts, lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int part = __builtin_amdgcn_readfirstlane(blockIdx.x % groups * kParts + wave / W);
    const int from = wave % W * kMine;
    const bool drafted = blockIdx.x / groups >= (uint32_t)a.n;
    const int row = blockIdx.x / groups - (drafted ? a.n : 0);
    f4_t l[kMine];
    const void *x = drafted ? row_of<F16>(a.drafted, row, a.drafted_stride)
                            : row_of<F16>(a.logits, row, a.stride);
    if (!drafted) load_part<F16>(l, x, part, a.vocab, from);
    fill_table(table);
    Span sp;
    if (!span_of(a, holder(a, row), sp) || row < sp.first || row > sp.last) return;
    const float heat = heat_of(a, sp.s);
    const bool cold = !(heat > 0.0f);
    if (drafted && (row == sp.last || cold)) return;
    if (drafted) load_part<F16>(l, x, part, a.vocab, from);
    const int draft = row < sp.last ? a.tokens[row + 1] : -1;
    __syncthreads();
    if (part >= parts) return;  // (waves that share no part)
    const int base = part * kPart + from * 256 + lane * 4;
    const bool judged = !cold && draft >= part * kPart && draft < min(part * kPart + kPart, a.vocab);
    float its = -INFINITY;
    if (judged) {
        its = load1<F16>(x, draft);
        if (!a.drafted) {
            const int at = draft - base;
#pragma unroll
            for (int i = 0; i < kMine; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) l[i][e] = at == i * 256 + e ? -INFINITY : l[i][e];
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMine; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = larger(top, l[i][e]);
    top = wave_max(top);
    if (W > 1) {
        if (lane == 0) tops[wave] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) top = larger(top, tops[i]);
    }
    Stat st = {0.0, top, judged ? __builtin_bit_cast(int, its) : INT32_MAX};
    if (!(larger(top, its) <= FLT_MAX)) {
        st.sum = NAN;
    } else if (top == -INFINITY) {
    } else if (cold) {
        // (read again: a loop that is not unrolled, beside the one that is)
        int first = INT32_MAX;
#pragma nounroll
        for (int i = kMine; i-- > 0;) {
            const f4_t again = load4<F16>(x, base + i * 256, a.vocab);
#pragma unroll
            for (int e = 4; e-- > 0;)
                if (again[e] == top) first = base + i * 256 + e;
        }
        st.at = wave_min(first);
        if (W > 1) {
            if (lane == 0) firsts[wave] = st.at;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < W; ++i) st.at = min(st.at, firsts[i]);
        }
    } else {
        const Power power(table, heat);
        const double m = top;
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < 4 * kMine; i += 2) {
            const double d[2] = {(double)l[i / 4][i % 4] - m, (double)l[i / 4][i % 4 + 1] - m};
            double w[2];
            power.of(d, w);
            sum += w[0];
            sum += w[1];
            __builtin_amdgcn_sched_barrier(0);  // else all are formed side by side
        }
        sum = wave_sum(sum);
        if (W > 1) {
            if (lane == 0) sums[wave] = sum;
            __syncthreads();
            sum = 0.0;
#pragma unroll
            for (int i = 0; i < W; ++i) sum += sums[i];
        }
        st.sum = sum;  // (of 1 and more)
    }
    if (lane == 0 && wave % W == 0) stats[(row + (drafted ? (int64_t)a.n : 0)) * parts + part] = st;
}

// ---- the refused draft ------------------------------------------------------
// A row's distribution: largest logit (`its`, the judged draft's, included), its first
// token, total weight (without the draft's where stats left it out); `fine` if it is one.
struct Whole {
    double sum;
    float top;
    int at;
    bool fine;
};
struct Parts {
    Stat of[kHeld];  // lane's parts: lane, lane + 64
    __device__ __forceinline__ void load(const Stat *stats, int parts) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int part = 64 * i + (int)(threadIdx.x % 64);
            of[i] = {0.0, -INFINITY, INT32_MAX};
            if (part < parts) of[i] = stats[part];
        }
    }
};
// By all lanes of a wave.
__device__ __forceinline__ Whole whole_of(const Stat *stats, const Parts &held, int parts,
                                          bool cold, const Power &power, float its) {
    const int lane = threadIdx.x % 64;
    Whole w = {0.0, its, INT32_MAX, true};
#pragma unroll
    for (int i = 0; i < kHeld; ++i) w.top = larger(w.top, held.of[i].top);
    for (int i = lane + 64 * kHeld; i < parts; i += 64) w.top = larger(w.top, stats[i].top);
    w.top = wave_max(w.top);
    const auto add = [&](const Stat &st) {
        if (st.sum != st.sum) w.fine = false;
        if (st.top == w.top) w.at = min(w.at, st.at);
        if (!cold) w.sum += st.sum * power.exact((double)st.top - (double)w.top);
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) add(held.of[i]);
    for (int i = lane + 64 * kHeld; i < parts; i += 64) add(stats[i]);
    if (cold)
        w.at = wave_min(w.at);
    else
        w.sum = wave_sum(w.sum);
    w.fine = __all(w.fine) && w.top != -INFINITY;
    return w;
}
// The judged draft's logit, minus infinity for a token outside the vocabulary.
__device__ __forceinline__ float drafted_logit(const Stat *stats, const Parts &held, int draft,
                                               bool real) {
    if (!real) return -INFINITY;
    const int part = draft / kPart;
    int at;
    if (part < 64 * kHeld)
        at = __builtin_amdgcn_readlane(part < 64 ? held.of[0].at : held.of[1].at, part % 64);
    else
        at = stats[part].at;
    return __builtin_bit_cast(float, at);
}

// The first row of the conversation whose draft is refused (its last row, if none
// is), and what follows.  Each of the workgroup's waves takes a row.
__device__ __forceinline__ Verdict judge(const VerifyArgs &a, const Stat *stats, int parts,
                                         const Span &sp, float heat, const Power &power,
                                         Verdict (&seen)[kPickWaves]) {
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const bool cold = !(heat > 0.0f);
    for (int row0 = sp.first;; row0 += kPickWaves) {
        const int row = row0 + wave;
        Verdict v = {0.0, 0.0, 0.0f, 0.0f, 0.0f, row, -1, -1, 0};
        Parts of_p, of_q;
        const Stat *ps = stats + (int64_t)row * parts;
        const Stat *qs = stats + ((int64_t)a.n + row) * parts;
        const bool last = row == sp.last, drafted = a.drafted && !last && !cold;
        float u = 0.0f;
        if (row <= sp.last) {
            of_p.load(ps, parts);
            if (drafted) of_q.load(qs, parts);
            u = a.uniform[2 * (int64_t)row];
            v.u = a.uniform[2 * (int64_t)row + 1];
            if (!last) v.draft = __builtin_amdgcn_readfirstlane(a.tokens[row + 1]);
        }
        __syncthreads();  // (the table, in the first round)
        if (row <= sp.last) {
            const bool real = v.draft >= 0 && v.draft < a.vocab;
            const float its = drafted_logit(ps, of_p, v.draft, real && !cold);
            const Whole p = whole_of(ps, of_p, parts, cold, power, its);
            v.p_top = p.top;
            v.at = p.at;
            if (!p.fine) {
                v.how = kNone;
            } else if (cold) {
                if (last || v.draft != p.at) v.how = kGreedy;
            } else {
                const double wd = power.exact((double)its - (double)p.top);
                v.p_share = 1.0 / (p.sum + (a.drafted ? 0.0 : wd));
                if (last) {
                    v.how = kPlain;
                } else if (!drafted) {
                    if (!((double)u < wd * v.p_share)) v.how = real ? kWithout : kPlain;
                } else {
                    const float its_q = drafted_logit(qs, of_q, v.draft, real);
                    const Whole q = whole_of(qs, of_q, parts, false, power, its_q);
                    v.q_top = q.top;
                    v.q_share = 1.0 / q.sum;
                    const double qd = power.exact((double)its_q - (double)q.top) * v.q_share;
                    if (!q.fine)
                        v.how = kNone;
                    else if (!((double)u * qd < wd * v.p_share))
                        v.how = kRest;
                }
            }
        }
        if (lane == 0) seen[wave] = v;
        __syncthreads();
        int found = -1;
#pragma unroll
        for (int i = kPickWaves; i-- > 0;)
            if (row0 + i <= sp.last && seen[i].how >= 0) found = i;
        if (found >= 0) return seen[found];
    }
}

__global__ __launch_bounds__(kPickThreads) void judge_kernel(VerifyArgs a, const Stat *stats,
                                                             Verdict *verdicts, int parts) {
    __shared__ double table[256];
    __shared__ Verdict seen[kPickWaves];
    const float heat = heat_of(a, blockIdx.x);
    Span sp;
    if (!span_of(a, blockIdx.x, sp)) return;
    fill_table(table);
    const Verdict v = judge(a, stats, parts, sp, heat, Power(table, heat), seen);
    if (threadIdx.x == 0) verdicts[sp.s] = v;
}

// max(p - q, 0) of a token.  Two products, each rounded, then the difference: as one
// fused operation equal p and q would leave the rounding of one of them.
__device__ __forceinline__ double above(double p, double p_share, double q, double q_share) {
#pragma clang fp contract(off)
    return fmax(p * p_share - q * q_share, 0.0);
}

// Sums of max(p - q, 0), a part to a workgroup, whose waves take a load each of p and
// of q: a chain as short as it gets (the whole call, a part to a wave and so, us: 12
// conversations over 32003 tokens 23.5 and 17.3, of 151936 29.8 and 26.6; 64 of them 73
// and 68).  Parts fastest in the grid: 64 conversations' 12.8 us, the other way 17.2.
// JUDGED: the verdicts are there; else every workgroup judges its conversation, and its
// first one notes the verdict.
template <bool F16, bool JUDGED>
__global__ __launch_bounds__(kPickThreads) void rest_kernel(VerifyArgs a, const Stat *stats,
                                                            Verdict *verdicts, double *rests,
                                                            int parts) {
    static_assert(kLoads == kPickWaves, "a load to a wave");
    __shared__ double table[256];
    __shared__ double sums[kPickWaves];
    __shared__ Verdict seen[kPickWaves];
    const int part = blockIdx.x, s = blockIdx.z * gridDim.y + blockIdx.y;
    if (s >= a.batch) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    Verdict v;
    if (JUDGED) v = verdicts[s];  // (of an empty conversation: whatever is there)
    const float heat = heat_of(a, s);
    const Power power(table, heat);
    Span sp;
    const bool some = span_of(a, s, sp);
    fill_table(table);
    if (!some) return;
    if (!JUDGED) {
        v = judge(a, stats, parts, sp, heat, power, seen);
        if (part == 0 && threadIdx.x == 0) verdicts[s] = v;
    }
    if (v.how != kRest) return;
    f4_t l[1], g[1];
    load_part<F16>(l, row_of<F16>(a.logits, v.row, a.stride), part, a.vocab, wave);
    load_part<F16>(g, row_of<F16>(a.drafted, v.row, a.drafted_stride), part, a.vocab, wave);
    __syncthreads();
    double d[8], w[8], sum = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        d[e] = (double)l[0][e] - (double)v.p_top;
        d[4 + e] = (double)g[0][e] - (double)v.q_top;
    }
    power.exact(d, w);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += above(w[e], v.p_share, w[4 + e], v.q_share);
    sum = wave_sum(sum);
    if (threadIdx.x % 64 == 0) sums[wave] = sum;
    __syncthreads();
    if (threadIdx.x != 0) return;
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < kPickWaves; ++i) sum += sums[i];
    rests[(int64_t)s * parts + part] = sum;
}

// ---- the next token ---------------------------------------------------------
// JUDGED: verdicts and rests are there.
template <bool F16, bool JUDGED>
__global__ __launch_bounds__(kPickThreads) void pick_kernel(VerifyArgs a, const Stat *stats,
                                                            const Verdict *verdicts,
                                                            const double *rests, int parts) {
    constexpr int kEach = kPart / kPickThreads;
    static_assert(kEach == 4, "one load to a thread");
    __shared__ double table[256];
    __shared__ double sums[kPickWaves];
    __shared__ Verdict seen[kPickWaves];
    __shared__ int highest;
    const int s = blockIdx.x, lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    // what depends on the conversation's number alone is requested together
    const float heat = heat_of(a, s);
    const Power power(table, heat);
    Verdict v;
    double held[kHeld] = {0.0, 0.0};
    if (JUDGED) {
        v = verdicts[s];
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (lane + 64 * i < parts) held[i] = rests[(int64_t)s * parts + lane + 64 * i];
    }
    Span sp;
    const bool some = span_of(a, s, sp);
    fill_table(table);
    if (!some) {
        if (threadIdx.x == 0) a.accepted[s] = 0, a.next[s] = -1;
        return;
    }
    if (!JUDGED) v = judge(a, stats, parts, sp, heat, power, seen);
    if (threadIdx.x == 0) {
        a.accepted[s] = v.row - sp.first;
        if (v.how == kNone) a.next[s] = -1;
        if (v.how == kGreedy) a.next[s] = v.at;
        highest = -1;
    }
    if (v.how == kNone || v.how == kGreedy) return;
    __syncthreads();  // (the table)
    // Shares of the parts, by every wave alike, 64 at a time: the held ones, then
    // those of a longer row.
    const auto share = [&](int i) -> double {
        const int part = 64 * i + lane;
        if (i < kHeld) return i == 0 ? held[0] : held[kHeld - 1];
        if (part >= parts) return 0.0;
        if (v.how == kRest) return rests[(int64_t)s * parts + part];
        const Stat st = stats[(int64_t)v.row * parts + part];
        return st.sum * power.exact((double)st.top - (double)v.p_top);
    };
    const int rounds = (parts + 63) / 64;
    double total;
    const auto add_up = [&] {
        total = held[0] + held[1];
        for (int i = kHeld; i < rounds; ++i) total += share(i);
        total = wave_sum(total);
    };
    if (JUDGED && v.how == kRest) {
        add_up();
        // rounding has left nothing above the draft's: all of p
        if (!(total > 0.0)) v.how = kPlain;
    }
    if (v.how != kRest) {
        Parts of;
        of.load(stats + (int64_t)v.row * parts, parts);
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            held[i] = of.of[i].sum * power.exact((double)of.of[i].top - (double)v.p_top);
        add_up();
    }
    if (v.how == kWithout && !(total > 0.0)) {
        if (threadIdx.x == 0) a.next[s] = v.draft;
        return;
    }
    // the first part that passes the target, or the last that holds a token
    const double target = (double)v.u * total;
    double below = 0.0, run = 0.0;
    int part = 0;
    for (int i = 0; i < rounds; ++i) {
        const double x = share(i), sum = up_to(x);
        const uint64_t holds = __ballot(x > 0.0);
        const uint64_t over = __ballot(run + sum > target) & holds;
        if (holds) {
            const int at = over ? __ffsll((unsigned long long)over) - 1 : 63 - __clzll(holds);
            part = 64 * i + at;
            below = run + (at ? lane_of(sum, at - 1) : 0.0);
        }
        if (over) break;
        run += lane_of(sum, 63);
    }
    // a thread's four neighbouring tokens, as weights
    const int first = part * kPart + threadIdx.x * kEach;
    const f4_t l = load4<F16>(row_of<F16>(a.logits, v.row, a.stride), first, a.vocab);
    f4_t g = l;
    if (JUDGED && v.how == kRest)
        g = load4<F16>(row_of<F16>(a.drafted, v.row, a.drafted_stride), first, a.vocab);
    double w[kEach], mine = 0.0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        w[i] = power.exact((double)l[i] - (double)v.p_top);
        if (JUDGED && v.how == kRest)
            w[i] = above(w[i], v.p_share, power.exact((double)g[i] - (double)v.q_top), v.q_share);
        if (v.how == kWithout && first + i == v.draft) w[i] = 0.0;
        mine += w[i];
    }
    const double upto = up_to(mine);
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    double at = below;
    int taken = -1;  // the wave that passes the target
    double start = 0.0;
#pragma unroll
    for (int i = 0; i < kPickWaves; ++i) {
        if (i == wave) start = at;
        at += sums[i];
        if (taken < 0 && sums[i] > 0.0 && at > target) taken = i;
    }
    int last = -1;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (w[i] > 0.0) last = first + i;
    if (taken < 0) {  // none does: the highest token of the part
        if (last >= 0) atomicMax(&highest, last);
        __syncthreads();
        if (threadIdx.x == 0) a.next[s] = highest;
        return;
    }
    if (wave != taken) return;
    // the first lane that passes it, and its first token that does (its last, where
    // the sums' rounding leaves none)
    const uint64_t holds = __ballot(last >= 0);
    const uint64_t over = __ballot(start + upto > target) & holds;
    const int lead = over ? __ffsll((unsigned long long)over) - 1 : 63 - __clzll(holds);
    if (lane != lead) return;
    at = start + (upto - mine);
    int token = last;
#pragma unroll
    for (int i = kEach; i-- > 0;) {
        double sum = at;
#pragma unroll
        for (int e = 0; e <= i; ++e) sum += w[e];
        if (w[i] > 0.0 && sum > target) token = first + i;
    }
    a.next[s] = token;
}

int parts_of(int64_t vocab) { return (int)((vocab + kPart - 1) / kPart); }

// The workspace: stats, then (with draft logits) verdicts and rests.
struct Shares {
    size_t verdicts, rests, bytes;
};
Shares shares_of(int64_t n, int64_t batch, int64_t vocab, bool drafted) {
    const size_t parts = (size_t)parts_of(vocab);
    Shares sh = {(size_t)n * (drafted ? 2u : 1u) * parts * sizeof(Stat), 0, 0};
    sh.rests = sh.verdicts + (drafted ? (size_t)batch * sizeof(Verdict) : 0);
    sh.bytes = sh.rests + (drafted ? (size_t)batch * parts * sizeof(double) : 0);
    return sh;
}

template <bool F16>
hipError_t run(const VerifyArgs &a, void *ws, hipStream_t stream) {
    const int parts = parts_of(a.vocab);
    const Shares sh = shares_of(a.n, a.batch, a.vocab, a.drafted != nullptr);
    const int64_t rows = (int64_t)a.n * (a.drafted ? 2 : 1);
    Stat *stats = (Stat *)ws;
    Verdict *verdicts = (Verdict *)((uint8_t *)ws + sh.verdicts);
    double *rests = (double *)((uint8_t *)ws + sh.rests);
    const int64_t cus = device_shape().cus;
    const int64_t many = rows * ((parts + kWaves - 1) / kWaves);
    const dim3 batch((uint32_t)a.batch);
    const uint32_t across = a.batch < 32768 ? (uint32_t)a.batch : 32768u;
    // (whole calls, us, a part to a wave and to four: rows of 151936 tokens without draft
    // logits, four 9.9 and 8.4, 16 11.2 and 9.9, 32 12.9 and 12.2, 64 17.3 and 18.2, 256
    // 35.6 and 41.9; rows of 32003 with draft logits, 8 16.0 and 13.9, 64 17.5 and 17.0,
    // 96 19.0 and 18.9, 256 28.1 and 31.4)
    if (rows * parts <= 8 * cus)
        hipLaunchKernelGGL((stats_kernel<F16, kWaves>), dim3((uint32_t)(rows * parts)),
                           dim3(kThreads), 0, stream, a, stats, parts);
    else
        hipLaunchKernelGGL((stats_kernel<F16, 1>), dim3((uint32_t)many), dim3(kThreads), 0,
                           stream, a, stats, parts);
    if (!a.drafted) {
        hipLaunchKernelGGL((pick_kernel<F16, false>), batch, dim3(kPickThreads), 0, stream, a,
                           stats, nullptr, nullptr, parts);
        return hipGetLastError();
    }
    const dim3 all((uint32_t)parts, across, ((uint32_t)a.batch + across - 1) / across);
    // As many parts as run at once: every workgroup of rest judges its conversation, a
    // launch less (whole calls of four rows a conversation, us, so and with a launch of
    // their own: over 32003 tokens 7 conversations 13.8 and 15.4, 32 19.7 and 21.0, 48
    // 25.1 and 24.0; over 151936 four 15.2 and 16.8, 12 27.3 and 26.8, 64 83 and 64)
    if ((int64_t)a.batch * parts <= 2 * cus) {
        hipLaunchKernelGGL((rest_kernel<F16, false>), all, dim3(kPickThreads), 0, stream, a, stats,
                           verdicts, rests, parts);
    } else {
        hipLaunchKernelGGL(judge_kernel, batch, dim3(kPickThreads), 0, stream, a, stats, verdicts,
                           parts);
        hipLaunchKernelGGL((rest_kernel<F16, true>), all, dim3(kPickThreads), 0, stream, a, stats,
                           verdicts, rests, parts);
    }
    hipLaunchKernelGGL((pick_kernel<F16, true>), batch, dim3(kPickThreads), 0, stream, a, stats,
                       verdicts, rests, parts);
    return hipGetLastError();
}

}  // namespace

size_t verify_workspace_bytes(int64_t n, int64_t batch, int64_t vocab, bool drafted) {
    return shares_of(n, batch, vocab, drafted).bytes;
}

hipError_t launch_verify(const VerifyArgs &a, int x_f16, void *ws, hipStream_t stream) {
    return x_f16 ? run<true>(a, ws, stream) : run<false>(a, ws, stream);
}

}  // namespace q4
