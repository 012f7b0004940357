// Append to the paged key/value cache: per-head norms and position rotation of
// q and k on the way, v converted, one pass over the rows.
//
// A group of LPH lanes holds one head row of dim elements, 8 to a lane, as two
// runs of four: the two halves of four rotation pairs (split-half order), four
// whole pairs (interleaved order), or eight elements that pass unrotated.  The
// rotation is then arithmetic inside a lane, and the norm's sum of squares a
// reduction over the group.  The angles depend on the token and the lane alone,
// so a group that walks several heads of its token forms sine and cosine once.
//
// Bound by the bytes: 8191 tokens of 16 + 2 x 8 heads of 256, binary16, in
// 56.5 us: 4.8 TB/s, where a copy of as many bytes reaches 4.8 to 5.4.  A single
// token (32 + 2 x 8 heads of 128) takes 3.3 us, one launch.
//
// Into a cache of codes a row of K or V needs its largest magnitude, from the same
// reduction over the group, and goes out as codes x / s rounded to even with s = max
// |x| / 127.  That is bound by its arithmetic (the sines, and a correctly rounded
// quotient an element): the 8191 tokens above, half of each head rotated, in 52 us,
// 4.5 TB/s of its bytes (58 us with the library's division and sine); a single
// token in 3.7 us.
#include <float.h>

#include "q4_0_device.h"
#include "q4_0_internal.h"

namespace q4 {

namespace {

constexpr int kThreads = 256;
typedef _Float16 h4_t __attribute__((ext_vector_type(4)));

template <bool F16> __device__ __forceinline__ f4_t load4(const void *p, int64_t at) {
    if (F16) {
        const h4_t h = *(const h4_t *)((const _Float16 *)p + at);
        return f4_t{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
    }
    return *(const f4_t *)((const float *)p + at);
}

template <bool F16> __device__ __forceinline__ void store4(void *p, int64_t at, f4_t x) {
    if (F16)
        *(h4_t *)((_Float16 *)p + at) =
            h4_t{(_Float16)x[0], (_Float16)x[1], (_Float16)x[2], (_Float16)x[3]};
    else
        *(f4_t *)((float *)p + at) = x;
}

// Sine and cosine of position * inv_freq.  The product and its reduction to
// one turn are formed in float64 (a float32 angle of a position of 10^5 is off
// by 0.004 already); what is left lies in [-pi, pi] and float32 carries it.
__device__ __forceinline__ void turn(int position, float inv_freq, float *s, float *c) {
    const double angle = (double)position * (double)inv_freq;
    const double n = rint(angle * 0.15915494309189533577);
    const double r = fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586477, angle));
    sincosf((float)r, s, c);
}

// The same by quarter turns: what is left lies in [-pi/4, pi/4], where the series of
// sine and cosine need five and six terms (2^-29 at most is left out).  A third of the
// library function's operations, which an append in 8 bits, bound by its
// arithmetic, has to spare; the binary16 append, bound by its bytes, has not.  Nor does
// it cost accuracy: rms 1.5e-8 and 1.9e-8 (of the sine, the cosine), where an exact
// function of an angle rounded in [-pi, pi] is 3.8e-8 off; so the two appends' q_out may
// differ by a step of float32.
__device__ __forceinline__ void quarter_turn(int position, float inv_freq, float *s, float *c) {
    const double angle = (double)position * (double)inv_freq;
    const double magic = 6755399441055744.0;  // 1.5 2^52: the sum's low bits are the integer
    const double k = fma(angle, 0.63661977236758134308, magic);
    const double n = k - magic;
    const float r =
        (float)fma(-n, 6.123233995736766e-17, fma(-n, 1.5707963267948965580, angle));
    const int q = (int)(uint32_t)__builtin_bit_cast(uint64_t, k);
    const float z = r * r;
    const float sn =
        fmaf(r * z, fmaf(z, fmaf(z, fmaf(z, 2.7557319e-6f, -1.9841270e-4f), 8.3333333e-3f),
                         -1.6666667e-1f), r);
    const float cs = fmaf(
        z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.7557319e-7f, 2.4801587e-5f), -1.3888889e-3f),
                        4.1666667e-2f), -0.5f), 1.0f);
    const float a = q & 1 ? cs : sn, b = q & 1 ? sn : cs;
    *s = q & 2 ? -a : a;
    *c = (q + 1) & 2 ? -b : b;
}

// Four elements as codes of scale `s`, one word; `r` is 1 / s, correctly rounded.
// The quotient is the product with r corrected twice by its exact remainder, which
// is the correctly rounded quotient (s is kept where no remainder is subnormal).  It
// is rounded by an addition that leaves the whole number in the low bits.
__device__ __forceinline__ uint32_t codes_of(f4_t x, float s, float r) {
    uint32_t t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float q = x[i] * r;
        q = fmaf(fmaf(-q, s, x[i]), r, q);
        q = fmaf(fmaf(-q, s, x[i]), r, q);
        t[i] = __builtin_bit_cast(uint32_t, q + 12582912.0f);
    }
    return __builtin_amdgcn_perm(t[1], t[0], 0x0C0C0400u) |
           __builtin_amdgcn_perm(t[3], t[2], 0x04000C0Cu);
}

template <bool XF16, bool QF16, bool CODES, int LPH>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a, int chunks) {
    constexpr int kGroups = kThreads / LPH;
    const int dim = a.cache.dim;
    const int64_t t = blockIdx.x / chunks;
    const int chunk = blockIdx.x % chunks;
    const int j = threadIdx.x % LPH;
    const int heads = a.cache.heads;
    const int total = a.q_heads + 2 * heads;
    const bool active = 8 * j < dim;
    const bool rotated = 8 * j < a.rot_dim;
    // the lane's two runs of four elements
    const bool split = rotated && !a.interleaved;
    const int e0 = split ? 4 * j : 8 * j;
    const int e1 = split ? 4 * j + a.rot_dim / 2 : 8 * j + 4;
    float sn[4], cs[4];
    if (rotated) {
        const int p = a.positions[t];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (CODES)
                quarter_turn(p, a.inv_freq[4 * j + i], &sn[i], &cs[i]);
            else
                turn(p, a.inv_freq[4 * j + i], &sn[i], &cs[i]);
            sn[i] *= a.amplitude;
            cs[i] *= a.amplitude;
        }
    }
    const int64_t slot = a.slots[t];
    const int shift = a.cache.page_shift;
    const bool kept = slot >= 0 && slot < (a.cache.pages << shift);
    const int64_t page = slot >> shift, off = slot & ((INT64_C(1) << shift) - 1);
    for (int h = chunk * kGroups + threadIdx.x / LPH; h < total; h += chunks * kGroups) {
        const bool is_q = h < a.q_heads;
        const bool is_v = h >= a.q_heads + heads;
        const int hh = is_q ? h : (is_v ? h - a.q_heads - heads : h - a.q_heads);
        const void *src = is_q ? a.q : (is_v ? a.v : a.k);
        const int64_t at =
            t * (is_q ? a.q_stride : (is_v ? a.v_stride : a.k_stride)) + (int64_t)hh * dim;
        f4_t x0 = {0.0f, 0.0f, 0.0f, 0.0f}, x1 = x0;
        if (active) {
            x0 = load4<XF16>(src, at + e0);
            x1 = load4<XF16>(src, at + e1);
        }
        const float *w = is_q ? a.q_norm : a.k_norm;
        if (!is_v && w) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) ss += x0[i] * x0[i] + x1[i] * x1[i];
#pragma unroll
            for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor(ss, m);
            const float r = 1.0f / sqrtf(ss / (float)dim + a.eps);
            if (active) {
                const f4_t w0 = *(const f4_t *)(w + e0), w1 = *(const f4_t *)(w + e1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x0[i] = x0[i] * r * (w0[i] + a.weight_offset);
                    x1[i] = x1[i] * r * (w1[i] + a.weight_offset);
                }
            }
        }
        if (!is_v && rotated) {
            if (split) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u = x0[i], v = x1[i];
                    x0[i] = u * cs[i] - v * sn[i];
                    x1[i] = v * cs[i] + u * sn[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float u = x0[2 * i], v = x0[2 * i + 1];
                    x0[2 * i] = u * cs[i] - v * sn[i];
                    x0[2 * i + 1] = v * cs[i] + u * sn[i];
                    const float y = x1[2 * i], z = x1[2 * i + 1];
                    x1[2 * i] = y * cs[2 + i] - z * sn[2 + i];
                    x1[2 * i + 1] = z * cs[2 + i] + y * sn[2 + i];
                }
            }
        }
        float step = 0.0f;
        if (CODES && !is_q) {
            // the row's largest magnitude, as bits: what is no number is larger
            // than every number
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = x0[i], v = x1[i];
                top = max(top, max(__builtin_bit_cast(uint32_t, u) & 0x7FFFFFFFu,
                                   __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu));
            }
#pragma unroll
            for (int m = 1; m < LPH; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
            step = __builtin_bit_cast(float, top) / 127.0f;
            if (step < FLT_MIN) step = 0.0f;  // its codes would need smaller steps than float32's
            if (top >= 0x7F800000u) step = NAN;
        }
        if (!active) continue;
        if (is_q) {
            const int64_t o = (t * a.q_heads + hh) * dim;
            store4<QF16>(a.q_out, o + e0, x0);
            store4<QF16>(a.q_out, o + e1, x1);
        } else if (CODES) {
            if (!kept) continue;
            const int64_t row = ((page * heads + hh) << shift) + off;
            uint8_t *dst = (uint8_t *)(is_v ? a.cache.v : a.cache.k) + row * dim;
            float s = step;
            if (s < 0x1p-60f) {  // (rarely) up to where remainders are exact
                s *= 0x1p64f;
                x0 *= 0x1p64f;
                x1 *= 0x1p64f;
            }
            const bool fine = s > 0.0f;
            const float r = fine ? 1.0f / s : 0.0f;
            *(uint32_t *)(dst + e0) = fine ? codes_of(x0, s, r) : 0u;
            *(uint32_t *)(dst + e1) = fine ? codes_of(x1, s, r) : 0u;
            if (j == 0) (is_v ? a.cache.v_scale : a.cache.k_scale)[row] = step;
        } else if (kept) {
            const int64_t o = (((page * heads + hh) << shift) + off) * dim;
            void *dst = is_v ? a.cache.v : a.cache.k;
            store4<true>(dst, o + e0, x0);
            store4<true>(dst, o + e1, x1);
        }
    }
}

template <bool XF16, bool QF16, bool CODES, int LPH>
hipError_t launch(const AppendArgs &a, hipStream_t stream) {
    const int groups = kThreads / LPH;
    const int total = a.q_heads + 2 * a.cache.heads;
    const int all = (total + groups - 1) / groups;
    // few tokens: one head per group, so the step is as short as one row;
    // enough tokens to fill the device: a workgroup walks its whole token, whose
    // angles it forms once.  Both ways (us; float32, binary16 alike): 32 + 2 x 8
    // heads of 128, 256 tokens 4.9 and 5.8, 400 tokens 6.5 and 6.5, 512 tokens
    // 7.4 and 6.7, 2048 tokens 19.6 and 17.4; 16 + 2 x 8 of 256, 256 tokens 5.7
    // and 6.5, 400 tokens 7.8 and 7.1; 64 + 2 x 8 of 64, 341 tokens 5.3 and 6.0,
    // 512 tokens 6.8 and 6.5.
    // In codes, where a row is more arithmetic: 32 + 2 x 8 heads of 128, 512 tokens 6.4
    // and 6.6, 640 tokens 7.4 and 7.4, 1024 tokens 10.0 and 8.8; 16 + 2 x 8 of 256,
    // 512 tokens 7.9 and 7.9, 640 tokens 9.2 and 9.0; 64 + 2 x 8 of 64, 640 tokens
    // 6.8 and 6.9, 1024 tokens 9.2 and 8.1.
    const int chunks = a.n * all <= (CODES ? 2048 : 1024) ? all : 1;
    hipLaunchKernelGGL((append_kernel<XF16, QF16, CODES, LPH>), dim3((uint32_t)(a.n * chunks)),
                       dim3(kThreads), 0, stream, a, chunks);
    return hipGetLastError();
}

template <bool XF16, bool QF16, bool CODES>
hipError_t by_dim(const AppendArgs &a, hipStream_t stream) {
    if (a.cache.dim <= 64) return launch<XF16, QF16, CODES, 8>(a, stream);
    if (a.cache.dim <= 128) return launch<XF16, QF16, CODES, 16>(a, stream);
    if (a.cache.dim <= 256) return launch<XF16, QF16, CODES, 32>(a, stream);
    return launch<XF16, QF16, CODES, 64>(a, stream);
}

template <bool CODES>
hipError_t by_type(const AppendArgs &a, int x_f16, int q_f16, hipStream_t stream) {
    if (x_f16)
        return q_f16 ? by_dim<true, true, CODES>(a, stream) : by_dim<true, false, CODES>(a, stream);
    return q_f16 ? by_dim<false, true, CODES>(a, stream) : by_dim<false, false, CODES>(a, stream);
}

// Rows of an 8-bit cache as numbers: a group of LPH lanes to a row, 8 codes to a
// lane; K in one half of the grid's second dimension, V in the other.  Bound by the
// bytes it writes: 8191 tokens of 2 x 8 heads of 256 as binary16 (67 MB, and 35 MB
// read) in 21 us, 4.8 TB/s.
template <bool YF16, int LPH>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadArgs a) {
    constexpr int kGroups = kThreads / LPH;
    const int dim = a.cache.dim, heads = a.cache.heads, shift = a.cache.page_shift;
    const bool is_v = blockIdx.y ? true : !a.k;
    const int j = threadIdx.x % LPH;
    if (8 * j >= dim) return;
    const float *scales = is_v ? a.cache.v_scale : a.cache.k_scale;
    const uint8_t *codes = (const uint8_t *)(is_v ? a.cache.v : a.cache.k) + 8 * j;
    void *y = is_v ? a.v : a.k;
    const int64_t total = a.n * heads, stride = (int64_t)gridDim.x * kGroups;
    for (int64_t at = (int64_t)blockIdx.x * kGroups + threadIdx.x / LPH; at < total; at += stride) {
        const int64_t slot = a.slots[at / heads];
        f4_t x0 = {0.0f, 0.0f, 0.0f, 0.0f}, x1 = x0;
        if (slot >= 0 && slot < (a.cache.pages << shift)) {
            const int64_t row = (((slot >> shift) * heads + at % heads) << shift) +
                                (slot & ((INT64_C(1) << shift) - 1));
            const float step = scales[row];
            const u2_t w = load_u2(codes + row * dim);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x0[i] = step * (float)(int8_t)(w[0] >> (8 * i));
                x1[i] = step * (float)(int8_t)(w[1] >> (8 * i));
            }
        }
        store4<YF16>(y, at * dim + 8 * j, x0);
        store4<YF16>(y, at * dim + 8 * j + 4, x1);
    }
}

template <bool YF16, int LPH> hipError_t read(const ReadArgs &a, hipStream_t stream) {
    const int64_t total = a.n * a.cache.heads;
    hipLaunchKernelGGL((read_kernel<YF16, LPH>),
                       dim3((uint32_t)grid_for(total, kThreads / LPH), a.k && a.v ? 2u : 1u),
                       dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

template <bool YF16> hipError_t read_by_dim(const ReadArgs &a, hipStream_t stream) {
    if (a.cache.dim <= 64) return read<YF16, 8>(a, stream);
    if (a.cache.dim <= 128) return read<YF16, 16>(a, stream);
    if (a.cache.dim <= 256) return read<YF16, 32>(a, stream);
    return read<YF16, 64>(a, stream);
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, int x_f16, int q_f16, hipStream_t stream) {
    return a.cache.k_scale ? by_type<true>(a, x_f16, q_f16, stream)
                           : by_type<false>(a, x_f16, q_f16, stream);
}

hipError_t launch_kv_read8(const ReadArgs &a, int y_f16, hipStream_t stream) {
    return y_f16 ? read_by_dim<true>(a, stream) : read_by_dim<false>(a, stream);
}

}  // namespace q4
