// Verification of drafted tokens against the target's probabilities.
//
// With p = softmax(l / T) of a row and q = softmax(g / T) of the draft's (all of q on
// the draft where there is none), draft d is taken iff u q(d) < p(d).  After the
// first one refused the next token is drawn from max(p - q, 0), after the last one
// from p: the lowest token whose cumulative weight passes u' times the total.
//
// A draw is a border among up to 10^5 shares, so weights and sums are 64-bit: the
// same token comes out whatever the order of the sums.  A weight 2^x is a table's
// entry (256 of them) times a polynomial of the third degree, off by 2e-13.
//
// Three launches.  stats: maximum and sum of every part of every row, one read.
// rest (with the draft's logits): each conversation's refused draft, and the sums of
// max(p - q, 0) over the parts of its row.  pick: the part, then the token.
#include <float.h>

#include "q4_0_device.h"
#include "q4_0_internal.h"

namespace q4 {

namespace {

typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
typedef f4_t f4_any_t __attribute__((aligned(4)));
typedef h4_t h4_any_t __attribute__((aligned(2)));

constexpr int kThreads = 256;
constexpr int kPart = 8192;               // tokens of a part
constexpr int kPickThreads = 1024;
constexpr int kMaxParts = (1 << 24) / kPart;
constexpr double kLog2e = 1.4426950408889634;

// A part of a row: its largest logit, the first token that has it, and the sum of
// its weights relative to that logit.  A sum that is no number: the part holds a
// logit that is NaN or plus infinity.
struct Stat {
    double sum;
    float top;
    int32_t at;
};

// 2^x for the weights, from a table of 2^(i / 256) in LDS.
struct Power {
    const double *table;
    double c, least;  // 256 log2(e) / T, and where weights are 0
    __device__ __forceinline__ Power(const double *t, double heat)
        : table(t), c(256.0 * kLog2e / heat), least(-256.0 * 1100.0 / (256.0 * kLog2e / heat)) {}
    // exp(d / T) of a difference d <= 0
    __device__ __forceinline__ double operator()(double d) const {
        const double magic = 6755399441055744.0;  // 1.5 2^52: the sum's low bits are the integer
        d = fmax(d, least);
        const double k = fma(d, c, magic);
        const double r = fma(d, c, -(k - magic));
        const int i = (int)(uint32_t)__builtin_bit_cast(uint64_t, k);
        // e^z, z = r ln(2) / 256, |z| < 0.00136
        const double z = fma(fma(fma(3.3083026805413713e-09, r, 3.6655655969101062e-06), r,
                                 0.0027076061740622863), r, 1.0);
        return __builtin_amdgcn_ldexp(table[i & 255] * z, i >> 8);
    }
};
__device__ __forceinline__ void fill_table(double *table) {
    if (threadIdx.x < 256) table[threadIdx.x] = exp2((double)threadIdx.x / 256.0);
}

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
template <bool F16>
__device__ __forceinline__ const void *row_of(const void *p, int64_t row, int64_t stride) {
    return (const uint8_t *)p + row * stride * (F16 ? 2 : 4);
}

template <typename T, typename F> __device__ __forceinline__ T over_wave(T x, F f) {
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) x = f(x, __shfl_xor(x, i));
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
template <bool F16>
__global__ __launch_bounds__(kThreads) void stats_kernel(VerifyArgs a, Stat *stats, int parts) {
    constexpr int kLoads = kPart / (4 * kThreads);
    __shared__ double table[256];
    __shared__ float tops[kThreads / 64];
    __shared__ double sums[kThreads / 64];
    __shared__ int firsts[kThreads / 64];
    const int part = blockIdx.x % parts;
    const bool drafted = blockIdx.x / parts >= (uint32_t)a.n;
    const int row = blockIdx.x / parts - (drafted ? a.n : 0);
    Span sp;
    if (!span_of(a, holder(a, row), sp) || row < sp.first || row > sp.last) return;
    const float heat = heat_of(a, sp.s);
    const bool cold = !(heat > 0.0f);
    if (drafted && (row == sp.last || cold)) return;
    const void *x = drafted ? row_of<F16>(a.drafted, row, a.drafted_stride)
                            : row_of<F16>(a.logits, row, a.stride);
    const int base = part * kPart + threadIdx.x * 4;
    f4_t l[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) l[i] = load4<F16>(x, base + i * 4 * kThreads, a.vocab);
    fill_table(table);
    float top = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            top = fmaxf(top, l[i][e]);
            bad |= !(l[i][e] <= FLT_MAX);
        }
    top = over_wave(top, [](float p, float q) { return fmaxf(p, q); });
    const int wave = threadIdx.x / 64;
    if (threadIdx.x % 64 == 0) tops[wave] = top;
    bad = __syncthreads_or(bad);
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) top = fmaxf(top, tops[i]);
    double sum = 0.0;
    int first = INT32_MAX;
    if (cold) {
#pragma unroll
        for (int i = kLoads; i-- > 0;)
#pragma unroll
            for (int e = 4; e-- > 0;)
                if (l[i][e] == top) first = base + i * 4 * kThreads + e;
        first = over_wave(first, [](int p, int q) { return min(p, q); });
    } else if (top != -INFINITY) {
        const Power power(table, heat);
        const double m = top;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += power((double)l[i][e] - m);
        sum = over_wave(sum, [](double p, double q) { return p + q; });
    }
    if (threadIdx.x % 64 == 0) sums[wave] = sum, firsts[wave] = first;
    __syncthreads();
    if (threadIdx.x != 0) return;
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) {
        sum += sums[i];
        first = min(first, firsts[i]);
    }
    stats[(int64_t)blockIdx.x] = {bad ? (double)NAN : sum, top, first};
}

// ---- the refused draft ------------------------------------------------------
// A row's distribution: largest logit, its first token, total weight; `fine` if it
// is one.
struct Whole {
    double sum;
    float top;
    int at;
    bool fine;
};
// By all lanes of a wave.
__device__ __forceinline__ Whole whole_of(const Stat *stats, int parts, double c) {
    const int lane = threadIdx.x % 64;
    Whole w = {0.0, -INFINITY, INT32_MAX, true};
    for (int i = lane; i < parts; i += 64) w.top = fmaxf(w.top, stats[i].top);
    w.top = over_wave(w.top, [](float p, float q) { return fmaxf(p, q); });
    for (int i = lane; i < parts; i += 64) {
        const Stat st = stats[i];
        if (st.sum != st.sum) w.fine = false;
        if (st.top == w.top) w.at = min(w.at, st.at);
        if (st.sum > 0.0) w.sum += st.sum * exp2(((double)st.top - (double)w.top) * c);
    }
    w.sum = over_wave(w.sum, [](double p, double q) { return p + q; });
    w.at = over_wave(w.at, [](int p, int q) { return min(p, q); });
    w.fine = __all(w.fine) && w.top != -INFINITY;
    return w;
}

// How the next token is found.
enum { kNone, kGreedy, kPlain, kWithout, kRest };
struct Verdict {
    int row, how, draft;
    Whole p, q;
};

// The first row of the conversation whose draft is refused (its last row, if none
// is), and what follows.  Each of the workgroup's waves takes a row.
template <bool F16, int WAVES>
__device__ __forceinline__ Verdict judge(const VerifyArgs &a, const Stat *stats, int parts,
                                         const Span &sp, float heat, Verdict (&seen)[WAVES]) {
    const int wave = threadIdx.x / 64;
    const bool cold = !(heat > 0.0f);
    const double c = kLog2e / (double)heat;
    for (int row0 = sp.first;; row0 += WAVES) {
        const int row = row0 + wave;
        Verdict v = {row, -1, -1, {}, {}};
        if (row <= sp.last) {
            v.p = whole_of(stats + (int64_t)row * parts, parts, c);
            v.draft = row < sp.last ? a.tokens[row + 1] : -1;
            const bool real = v.draft >= 0 && v.draft < a.vocab;
            if (!v.p.fine) {
                v.how = kNone;
            } else if (cold) {
                if (row == sp.last || v.draft != v.p.at) v.how = kGreedy;
            } else if (row == sp.last) {
                v.how = kPlain;
            } else {
                const double u = a.uniform[2 * (int64_t)row];
                const double pd =
                    !real ? 0.0
                          : exp2(((double)load1<F16>(row_of<F16>(a.logits, row, a.stride), v.draft) -
                                  (double)v.p.top) * c) / v.p.sum;
                double qd = 1.0;
                if (a.drafted) {
                    v.q = whole_of(stats + ((int64_t)a.n + row) * parts, parts, c);
                    qd = !real ? 0.0
                               : exp2(((double)load1<F16>(
                                           row_of<F16>(a.drafted, row, a.drafted_stride), v.draft) -
                                       (double)v.q.top) * c) / v.q.sum;
                }
                if (a.drafted && !v.q.fine)
                    v.how = kNone;
                else if (!(u * qd < pd))
                    v.how = a.drafted ? kRest : real ? kWithout : kPlain;
            }
        }
        if (threadIdx.x % 64 == 0) seen[wave] = v;
        __syncthreads();
        int found = -1;
#pragma unroll
        for (int i = WAVES; i-- > 0;)
            if (row0 + i <= sp.last && seen[i].how >= 0) found = i;
        if (found >= 0) return seen[found];
        __syncthreads();
    }
}

// max(p - q, 0) of a token
__device__ __forceinline__ double rest_of(const Power &power, const Verdict &v, float l, float g) {
    const double p = power((double)l - (double)v.p.top) / v.p.sum;
    const double q = power((double)g - (double)v.q.top) / v.q.sum;
    return fmax(p - q, 0.0);
}

template <bool F16>
__global__ __launch_bounds__(kThreads, 4) void rest_kernel(VerifyArgs a, const Stat *stats,
                                                        double *rests, int parts) {
    constexpr int kLoads = kPart / (4 * kThreads);
    __shared__ double table[256];
    __shared__ double sums[kThreads / 64];
    __shared__ Verdict seen[kThreads / 64];
    const int part = blockIdx.x % parts, s = blockIdx.x / parts;
    Span sp;
    if (!span_of(a, s, sp)) return;
    const float heat = heat_of(a, s);
    if (!(heat > 0.0f)) return;
    fill_table(table);
    const Verdict v = judge<F16>(a, stats, parts, sp, heat, seen);
    if (v.how != kRest) return;
    const void *x = row_of<F16>(a.logits, v.row, a.stride);
    const void *y = row_of<F16>(a.drafted, v.row, a.drafted_stride);
    const Power power(table, heat);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int at = part * kPart + (i * kThreads + threadIdx.x) * 4;
        const f4_t l = load4<F16>(x, at, a.vocab), g = load4<F16>(y, at, a.vocab);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += rest_of(power, v, l[e], g[e]);
    }
    sum = over_wave(sum, [](double p, double q) { return p + q; });
    if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = sum;
    __syncthreads();
    if (threadIdx.x != 0) return;
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) sum += sums[i];
    rests[blockIdx.x] = sum;
}

// ---- the next token ---------------------------------------------------------
// Sum of x over the workgroup before this thread; the total in `total`.
__device__ __forceinline__ double before(double x, double (&sums)[kPickThreads / 64],
                                         double &total) {
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    double run = x;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
        const double y = __shfl_up(run, i);
        if (lane >= i) run += y;
    }
    __syncthreads();
    if (lane == 63) sums[wave] = run;
    __syncthreads();
    double base = 0.0;
    total = 0.0;
#pragma unroll
    for (int i = 0; i < kPickThreads / 64; ++i) {
        if (i < wave) base += sums[i];
        total += sums[i];
    }
    return base + run - x;
}

template <bool F16>
__global__ __launch_bounds__(kPickThreads) void pick_kernel(VerifyArgs a, const Stat *stats,
                                                            const double *rests, int parts) {
    constexpr int kEach = kPart / kPickThreads;
    __shared__ double table[256];
    __shared__ double share[kMaxParts];
    __shared__ double sums[kPickThreads / 64];
    __shared__ Verdict seen[kPickThreads / 64];
    __shared__ int found, highest;
    const int s = blockIdx.x;
    Span sp;
    if (!span_of(a, s, sp)) {
        if (threadIdx.x == 0) a.accepted[s] = 0, a.next[s] = -1;
        return;
    }
    const float heat = heat_of(a, s);
    fill_table(table);
    Verdict v = judge<F16>(a, stats, parts, sp, heat, seen);
    if (threadIdx.x == 0) {
        a.accepted[s] = v.row - sp.first;
        if (v.how == kNone) a.next[s] = -1;
        if (v.how == kGreedy) a.next[s] = v.p.at;
    }
    if (v.how == kNone || v.how == kGreedy) return;
    const Power power(table, heat);
    const double c = kLog2e / (double)heat;
    const void *x = row_of<F16>(a.logits, v.row, a.stride);
    const void *y = a.drafted ? row_of<F16>(a.drafted, v.row, a.drafted_stride) : nullptr;
    // a thread's neighbouring tokens of a part, as weights
    double w[kEach];
    const auto weigh = [&](int part) {
        const int at = part * kPart + threadIdx.x * kEach;
#pragma unroll
        for (int i = 0; i < kEach; i += 4) {
            const f4_t l = load4<F16>(x, at + i, a.vocab);
            f4_t g = l;
            if (v.how == kRest) g = load4<F16>(y, at + i, a.vocab);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (v.how == kRest)
                    w[i + e] = rest_of(power, v, l[e], g[e]);
                else
                    w[i + e] = power((double)l[e] - (double)v.p.top);
                if (v.how == kWithout && at + i + e == v.draft) w[i + e] = 0.0;
            }
        }
    };
    const auto own_sum = [&]() {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) sum += w[i];
        return sum;
    };
    double total = 0.0;
    if (v.how == kRest) {
        for (int i = threadIdx.x; i < parts; i += kPickThreads)
            share[i] = rests[(int64_t)s * parts + i];
        __syncthreads();
        for (int i = 0; i < parts; ++i) total += share[i];
        // rounding has left nothing above the draft's: all of p
        if (!(total > 0.0)) v.how = kPlain;
        __syncthreads();
    }
    if (v.how != kRest) {
        const Stat *st = stats + (int64_t)v.row * parts;
        for (int i = threadIdx.x; i < parts; i += kPickThreads)
            share[i] = st[i].sum > 0.0
                           ? st[i].sum * exp2(((double)st[i].top - (double)v.p.top) * c)
                           : 0.0;
        __syncthreads();
        if (v.how == kWithout) {
            double sum;
            weigh(v.draft / kPart);
            before(own_sum(), sums, sum);
            if (threadIdx.x == 0) share[v.draft / kPart] = sum;
            __syncthreads();
        }
        total = 0.0;
        for (int i = 0; i < parts; ++i) total += share[i];
        if (v.how == kWithout && !(total > 0.0)) {  // the draft is all there is
            if (threadIdx.x == 0) a.next[s] = v.draft;
            return;
        }
    }
    const double target = (double)a.uniform[2 * (int64_t)v.row + 1] * total;
    // the first part that passes the target, or the last that holds a token
    int part = 0;
    double below = 0.0, run = 0.0;
    for (int i = 0; i < parts; ++i) {
        if (!(share[i] > 0.0)) continue;
        part = i, below = run;
        run += share[i];
        if (run > target) break;
    }
    if (threadIdx.x == 0) found = INT32_MAX, highest = -1;
    weigh(part);
    double all;
    double at = below + before(own_sum(), sums, all);
    const int first = part * kPart + threadIdx.x * kEach;
    int mine = INT32_MAX, last = -1;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (!(w[i] > 0.0)) continue;
        at += w[i];
        last = first + i;
        if (mine == INT32_MAX && at > target) mine = first + i;
    }
    if (mine != INT32_MAX) atomicMin(&found, mine);
    if (last >= 0) atomicMax(&highest, last);
    __syncthreads();
    if (threadIdx.x == 0) a.next[s] = found != INT32_MAX ? found : highest;
}

int parts_of(int64_t vocab) { return (int)((vocab + kPart - 1) / kPart); }

template <bool F16>
hipError_t run(const VerifyArgs &a, void *ws, hipStream_t stream) {
    const int parts = parts_of(a.vocab);
    const int64_t rows = (int64_t)a.n * (a.drafted ? 2 : 1);
    Stat *stats = (Stat *)ws;
    double *rests = (double *)(stats + rows * parts);
    hipLaunchKernelGGL((stats_kernel<F16>), dim3((uint32_t)(rows * parts)), dim3(kThreads), 0,
                       stream, a, stats, parts);
    if (a.drafted)
        hipLaunchKernelGGL((rest_kernel<F16>), dim3((uint32_t)((int64_t)a.batch * parts)),
                           dim3(kThreads), 0, stream, a, stats, rests, parts);
    hipLaunchKernelGGL((pick_kernel<F16>), dim3((uint32_t)a.batch), dim3(kPickThreads), 0, stream,
                       a, stats, rests, parts);
    return hipGetLastError();
}

}  // namespace

size_t verify_workspace_bytes(int64_t n, int64_t batch, int64_t vocab, bool drafted) {
    const size_t parts = (size_t)parts_of(vocab);
    return (size_t)n * (drafted ? 2u : 1u) * parts * sizeof(Stat) +
           (drafted ? (size_t)batch * parts * sizeof(double) : 0);
}

hipError_t launch_verify(const VerifyArgs &a, int x_f16, void *ws, hipStream_t stream) {
    return x_f16 ? run<true>(a, ws, stream) : run<false>(a, ws, stream);
}

}  // namespace q4
