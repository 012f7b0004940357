// Residual step: norm after a half block, gate, residual add, norm before the
// next, one pass over each row.
//
// A row stays in registers between its loads and its stores: W waves hold it,
// CH chunks of VEC elements to a lane, and the two sums of squares (of the
// block's output, then of the new residual) are reductions over those waves.
// Bound by the bytes of b, h, h_out and y, each read or written once: 16383 rows
// of 5120 (binary16 b and y) in 196 us, 5.1 TB/s, where a copy of as many bytes
// reaches 4.8 to 5.4; rows of 5119 take 4 % longer.  One row of 2560 takes
// 3.2 us, one launch.
#include "q4_0_device.h"
#include "q4_0_internal.h"

namespace q4 {

namespace {

typedef _Float16 h4_t __attribute__((ext_vector_type(4)));

// Four neighbouring elements of a row.  RAGGED rows start and end anywhere: the
// loads and stores then assume an element's alignment only (the hardware takes
// such addresses), and the row's last elements go one by one, zeros after them.
struct Chunk {
    float v[4];
};
typedef f4_t f4_any_t __attribute__((aligned(4)));
typedef h4_t h4_any_t __attribute__((aligned(2)));

template <bool RAGGED> __device__ __forceinline__ Chunk load_f32(const float *p, int i, int dim) {
    Chunk c;
    if (!RAGGED || i + 4 <= dim) {
        const f4_t x = RAGGED ? *(const f4_any_t *)(p + i) : *(const f4_t *)(p + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) c.v[k] = x[k];
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) c.v[k] = i + k < dim ? p[i + k] : 0.0f;
    }
    return c;
}

template <bool RAGGED, bool F16>
__device__ __forceinline__ Chunk load_x(const void *row, int64_t at, int i, int dim) {
    if (!F16) return load_f32<RAGGED>((const float *)row + at, i, dim);
    const _Float16 *p = (const _Float16 *)row + at;
    Chunk c;
    if (!RAGGED || i + 4 <= dim) {
        const h4_t x = RAGGED ? *(const h4_any_t *)(p + i) : *(const h4_t *)(p + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) c.v[k] = (float)x[k];
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) c.v[k] = i + k < dim ? (float)p[i + k] : 0.0f;
    }
    return c;
}

template <bool RAGGED, bool F16>
__device__ __forceinline__ void store_x(void *row, int64_t at, int i, int dim, const Chunk &c) {
    if (F16) {
        _Float16 *p = (_Float16 *)row + at;
        if (!RAGGED || i + 4 <= dim) {
            const h4_t x = {(_Float16)c.v[0], (_Float16)c.v[1], (_Float16)c.v[2],
                            (_Float16)c.v[3]};
            if (RAGGED)
                *(h4_any_t *)(p + i) = x;
            else
                *(h4_t *)(p + i) = x;
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (i + k < dim) p[i + k] = (_Float16)c.v[k];
        }
    } else {
        float *p = (float *)row + at;
        if (!RAGGED || i + 4 <= dim) {
            const f4_t x = {c.v[0], c.v[1], c.v[2], c.v[3]};
            if (RAGGED)
                *(f4_any_t *)(p + i) = x;
            else
                *(f4_t *)(p + i) = x;
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (i + k < dim) p[i + k] = c.v[k];
        }
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

template <int W, int CH, bool RAGGED, bool BF16, bool YF16>
__global__ __launch_bounds__(kBlock<W>) void norm_kernel(NormArgs a) {
    static_assert(W == 1 || kBlock<W> == 64 * W, "a workgroup holds one row, or one per wave");
    __shared__ float red[2][16];
    constexpr int kRows = kBlock<W> / (64 * W);
    const int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / (64 * W);
    const int first = threadIdx.x % (64 * W) * 4, dim = a.dim;
    constexpr int kStep = 64 * W * 4;
    if (W == 1 && t >= a.n) return;
    Chunk b[CH], h[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = c * kStep + first;
        if (i < dim) {
            h[c] = load_f32<RAGGED>(a.h + t * a.h_stride, i, dim);
            if (a.b) b[c] = load_x<RAGGED, BF16>(a.b, t * a.b_stride, i, dim);
        }
    }
    float ss = 0.0f;
    if (a.b) {
        float r = 1.0f;
        if (a.post) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (c * kStep + first < dim)
#pragma unroll
                    for (int k = 0; k < 4; ++k) ss += b[c].v[k] * b[c].v[k];
            r = 1.0f / sqrtf(row_sum<W>(ss, red[0]) / (float)dim + a.eps);
        }
        ss = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = c * kStep + first;
            if (i >= dim) continue;
            if (a.post) {
                const Chunk w = load_f32<RAGGED>(a.post, i, dim);
#pragma unroll
                for (int k = 0; k < 4; ++k) b[c].v[k] = b[c].v[k] * r * (w.v[k] + a.weight_offset);
            }
            if (a.gate) {
                const float *g = a.gate + t * a.gate_row;
                if (a.gate_col) {
                    const Chunk w = load_f32<RAGGED>(g, i, dim);
#pragma unroll
                    for (int k = 0; k < 4; ++k) b[c].v[k] *= w.v[k];
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) b[c].v[k] *= g[0];
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) h[c].v[k] += a.alpha * b[c].v[k];
            store_x<RAGGED, false>(a.h_out, t * a.h_stride, i, dim, h[c]);
        }
    }
    if (!a.y) return;
#pragma unroll
    for (int c = 0; c < CH; ++c)
        if (c * kStep + first < dim)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (!RAGGED || c * kStep + first + k < dim) ss += h[c].v[k] * h[c].v[k];
    const float r = 1.0f / sqrtf(row_sum<W>(ss, red[1]) / (float)dim + a.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = c * kStep + first;
        if (i >= dim) continue;
        const Chunk w = load_f32<RAGGED>(a.pre, i, dim);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[c].v[k] = h[c].v[k] * r * (w.v[k] + a.weight_offset);
        store_x<RAGGED, YF16>(a.y, t * a.y_stride, i, dim, h[c]);
    }
}

template <int W, int CH, bool RAGGED, bool BF16, bool YF16>
hipError_t run(const NormArgs &a, hipStream_t stream) {
    constexpr int rows = kBlock<W> / (64 * W);
    const int64_t grid = (a.n + rows - 1) / rows;
    hipLaunchKernelGGL((norm_kernel<W, CH, RAGGED, BF16, YF16>), dim3((uint32_t)grid),
                       dim3(kBlock<W>), 0, stream, a);
    return hipGetLastError();
}

// Waves per row: up to eight, two chunks a lane, so that a row's loads are all
// in flight at once and one row alone is short; then more chunks, and sixteen
// waves only for what eight cannot hold.  16383 binary16 rows (us): of 512 on one
// wave 19, on four 26; of 1024 on four 34, on eight 42; of 2048 on four 75, on
// eight 77 to 81; of 4096 on eight 147, on four 152, on sixteen 166; of 4608 on
// eight 167, on four 187, on sixteen 188; of 8192 on eight 293, on four 316, on
// sixteen 292.  One row gains by more waves (2048: 3.7 on four, 3.2 on eight;
// 5120: 4.4 on eight, 4.0 on sixteen), float32 rows of 5120 too (16383: 242 on
// eight, 230 on sixteen).
template <bool RAGGED, bool BF16, bool YF16>
hipError_t by_size(const NormArgs &a, hipStream_t stream) {
    const int lanes = (a.dim + 3) / 4;
    if (lanes <= 128) return run<1, 2, RAGGED, BF16, YF16>(a, stream);
    if (lanes <= 512) return run<4, 2, RAGGED, BF16, YF16>(a, stream);
    if (lanes <= 1024) return run<8, 2, RAGGED, BF16, YF16>(a, stream);
    if (lanes <= 2048) return run<8, 4, RAGGED, BF16, YF16>(a, stream);
    static_assert(kNormMaxDim == 16 * 64 * 4 * 8, "eight chunks hold the widest row");
    return run<16, 8, RAGGED, BF16, YF16>(a, stream);
}

template <bool BF16, bool YF16> hipError_t by_alignment(const NormArgs &a, hipStream_t stream) {
    // rows on the boundary of four elements throughout, or not
    const auto on = [](const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; };
    bool even = a.dim % 4 == 0 && a.h_stride % 4 == 0 && on(a.h, 16);
    if (a.b) {
        even = even && a.b_stride % 4 == 0 && on(a.b, BF16 ? 8 : 16) && on(a.h_out, 16) &&
               on(a.post, 16);
        if (a.gate && a.gate_col) even = even && a.gate_row % 4 == 0 && on(a.gate, 16);
    }
    if (a.y) even = even && a.y_stride % 4 == 0 && on(a.y, YF16 ? 8 : 16) && on(a.pre, 16);
    return even ? by_size<false, BF16, YF16>(a, stream) : by_size<true, BF16, YF16>(a, stream);
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs &a, int b_f16, int y_f16, hipStream_t stream) {
    if (b_f16)
        return y_f16 ? by_alignment<true, true>(a, stream) : by_alignment<true, false>(a, stream);
    return y_f16 ? by_alignment<false, true>(a, stream) : by_alignment<false, false>(a, stream);
}

}  // namespace q4
