// Residual step: norm after a half block, gate, residual add, norm before the
// next, one pass over each row.
//
// A row stays in registers between its loads and its stores: W waves hold it,
// CH chunks of VEC elements to a lane, and the two sums of squares (of the
// block's output, then of the new residual) are reductions over those waves.
// Bound by the bytes of b, h, h_out and y; everything is read and written once.
#include "q4_0_device.h"
#include "q4_0_internal.h"

namespace q4 {

namespace {

typedef _Float16 h4_t __attribute__((ext_vector_type(4)));

template <int VEC> struct Chunk {
    float v[VEC];
};

template <int VEC> __device__ __forceinline__ Chunk<VEC> load_f32(const float *p) {
    Chunk<VEC> c;
    if (VEC == 4) {
        const f4_t x = *(const f4_t *)p;
#pragma unroll
        for (int i = 0; i < VEC; ++i) c.v[i] = x[i];
    } else {
        c.v[0] = *p;
    }
    return c;
}

template <int VEC, bool F16> __device__ __forceinline__ Chunk<VEC> load_x(const void *p,
                                                                          int64_t at) {
    if (!F16) return load_f32<VEC>((const float *)p + at);
    Chunk<VEC> c;
    if (VEC == 4) {
        const h4_t x = *(const h4_t *)((const _Float16 *)p + at);
#pragma unroll
        for (int i = 0; i < VEC; ++i) c.v[i] = (float)x[i];
    } else {
        c.v[0] = (float)((const _Float16 *)p)[at];
    }
    return c;
}

template <int VEC, bool F16>
__device__ __forceinline__ void store_x(void *p, int64_t at, const Chunk<VEC> &c) {
    if (VEC == 4) {
        if (F16)
            *(h4_t *)((_Float16 *)p + at) = h4_t{(_Float16)c.v[0], (_Float16)c.v[1 % VEC],
                                                 (_Float16)c.v[2 % VEC], (_Float16)c.v[3 % VEC]};
        else
            *(f4_t *)((float *)p + at) =
                f4_t{c.v[0], c.v[1 % VEC], c.v[2 % VEC], c.v[3 % VEC]};
    } else if (F16) {
        ((_Float16 *)p)[at] = (_Float16)c.v[0];
    } else {
        ((float *)p)[at] = c.v[0];
    }
}

// Sum over the W waves that hold a row.  `red` holds one float per wave of
// the workgroup; every thread of the workgroup takes part.
template <int W> __device__ __forceinline__ float row_sum(float x, float *red) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m);
    if (W == 1) return x;
    const int wave = threadIdx.x / 64;
    if (threadIdx.x % 64 == 0) red[wave] = x;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) s += red[i];
    return s;
}

template <int W> constexpr int kBlock = W < 4 ? 256 : 64 * W;

template <int W, int CH, int VEC, bool BF16, bool YF16>
__global__ __launch_bounds__(kBlock<W>) void norm_kernel(NormArgs a) {
    static_assert(W == 1 || kBlock<W> == 64 * W, "a workgroup holds one row, or one per wave");
    __shared__ float red[2][16];
    constexpr int kRows = kBlock<W> / (64 * W);
    const int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / (64 * W);
    const int lane = threadIdx.x % (64 * W);
    if (W == 1 && t >= a.n) return;
    Chunk<VEC> b[CH], h[CH];
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = (c * 64 * W + lane) * VEC;
        if (i < a.dim) {
            h[c] = load_f32<VEC>(a.h + t * a.h_stride + i);
            if (a.b) b[c] = load_x<VEC, BF16>(a.b, t * a.b_stride + i);
        }
    }
    if (a.b) {
        float r = 1.0f;
        if (a.post) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if ((c * 64 * W + lane) * VEC < a.dim)
#pragma unroll
                    for (int k = 0; k < VEC; ++k) ss += b[c].v[k] * b[c].v[k];
            }
            r = 1.0f / sqrtf(row_sum<W>(ss, red[0]) / (float)a.dim + a.eps);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = (c * 64 * W + lane) * VEC;
            if (i < a.dim) {
                if (a.post) {
                    const Chunk<VEC> w = load_f32<VEC>(a.post + i);
#pragma unroll
                    for (int k = 0; k < VEC; ++k)
                        b[c].v[k] = b[c].v[k] * r * (w.v[k] + a.weight_offset);
                }
                if (a.gate) {
                    const float *g = a.gate + t * a.gate_row;
                    if (a.gate_col) {
                        const Chunk<VEC> w = load_f32<VEC>(g + i);
#pragma unroll
                        for (int k = 0; k < VEC; ++k) b[c].v[k] *= w.v[k];
                    } else {
#pragma unroll
                        for (int k = 0; k < VEC; ++k) b[c].v[k] *= g[0];
                    }
                }
#pragma unroll
                for (int k = 0; k < VEC; ++k) h[c].v[k] += a.alpha * b[c].v[k];
                store_x<VEC, false>(a.h_out, t * a.h_stride + i, h[c]);
            }
        }
    }
    if (!a.y) return;
    ss = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if ((c * 64 * W + lane) * VEC < a.dim)
#pragma unroll
            for (int k = 0; k < VEC; ++k) ss += h[c].v[k] * h[c].v[k];
    }
    const float r = 1.0f / sqrtf(row_sum<W>(ss, red[1]) / (float)a.dim + a.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = (c * 64 * W + lane) * VEC;
        if (i < a.dim) {
            const Chunk<VEC> w = load_f32<VEC>(a.pre + i);
#pragma unroll
            for (int k = 0; k < VEC; ++k) h[c].v[k] = h[c].v[k] * r * (w.v[k] + a.weight_offset);
            store_x<VEC, YF16>(a.y, t * a.y_stride + i, h[c]);
        }
    }
}

template <int W, int CH, int VEC, bool BF16, bool YF16>
hipError_t run(const NormArgs &a, hipStream_t stream) {
    constexpr int rows = kBlock<W> / (64 * W);
    const int64_t grid = (a.n + rows - 1) / rows;
    hipLaunchKernelGGL((norm_kernel<W, CH, VEC, BF16, YF16>), dim3((uint32_t)grid),
                       dim3(kBlock<W>), 0, stream, a);
    return hipGetLastError();
}

// Waves per row: the fewest that hold the row in two chunks a lane, so that a
// row's loads are all in flight at once; 16 waves and more chunks above.
template <int VEC, bool BF16, bool YF16>
hipError_t by_size(const NormArgs &a, hipStream_t stream) {
    const int64_t lanes = (a.dim + VEC - 1) / VEC;
    if (lanes <= 128) return run<1, 2, VEC, BF16, YF16>(a, stream);
    if (lanes <= 512) return run<4, 2, VEC, BF16, YF16>(a, stream);
    if (lanes <= 1024) return run<8, 2, VEC, BF16, YF16>(a, stream);
    if (lanes <= 2048) return run<16, 2, VEC, BF16, YF16>(a, stream);
    if (lanes <= 8192) return run<16, 8, VEC, BF16, YF16>(a, stream);
    return run<16, 32, VEC, BF16, YF16>(a, stream);
}

template <bool BF16, bool YF16> hipError_t by_alignment(const NormArgs &a, hipStream_t stream) {
    // four elements at a time where every row starts on their boundary
    const auto on = [](const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; };
    bool vec = a.dim % 4 == 0 && a.h_stride % 4 == 0 && on(a.h, 16);
    if (a.b) {
        vec = vec && a.b_stride % 4 == 0 && on(a.b, BF16 ? 8 : 16) && on(a.h_out, 16) &&
              on(a.post, 16);
        if (a.gate && a.gate_col) vec = vec && a.gate_row % 4 == 0 && on(a.gate, 16);
    }
    if (a.y) vec = vec && a.y_stride % 4 == 0 && on(a.y, YF16 ? 8 : 16) && on(a.pre, 16);
    return vec ? by_size<4, BF16, YF16>(a, stream) : by_size<1, BF16, YF16>(a, stream);
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs &a, int b_f16, int y_f16, hipStream_t stream) {
    if (b_f16) return y_f16 ? by_alignment<true, true>(a, stream) : by_alignment<true, false>(a, stream);
    return y_f16 ? by_alignment<false, true>(a, stream) : by_alignment<false, false>(a, stream);
}

}  // namespace q4
