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

template <bool XF16, bool QF16, int LPH>
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
        if (!active) continue;
        if (is_q) {
            const int64_t o = (t * a.q_heads + hh) * dim;
            store4<QF16>(a.q_out, o + e0, x0);
            store4<QF16>(a.q_out, o + e1, x1);
        } else if (kept) {
            const int64_t o = (((page * heads + hh) << shift) + off) * dim;
            _Float16 *dst = is_v ? a.cache.v : a.cache.k;
            store4<true>(dst, o + e0, x0);
            store4<true>(dst, o + e1, x1);
        }
    }
}

template <bool XF16, bool QF16, int LPH>
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
    const int chunks = a.n * all <= 1024 ? all : 1;
    hipLaunchKernelGGL((append_kernel<XF16, QF16, LPH>), dim3((uint32_t)(a.n * chunks)),
                       dim3(kThreads), 0, stream, a, chunks);
    return hipGetLastError();
}

template <bool XF16, bool QF16> hipError_t by_dim(const AppendArgs &a, hipStream_t stream) {
    if (a.cache.dim <= 64) return launch<XF16, QF16, 8>(a, stream);
    if (a.cache.dim <= 128) return launch<XF16, QF16, 16>(a, stream);
    if (a.cache.dim <= 256) return launch<XF16, QF16, 32>(a, stream);
    return launch<XF16, QF16, 64>(a, stream);
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, int x_f16, int q_f16, hipStream_t stream) {
    if (x_f16) return q_f16 ? by_dim<true, true>(a, stream) : by_dim<true, false>(a, stream);
    return q_f16 ? by_dim<false, true>(a, stream) : by_dim<false, false>(a, stream);
}

}  // namespace q4
