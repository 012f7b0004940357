// Lookup of rows of the repacked Q4_0 table, scaled, and the first block's norm.
//
// One workgroup to a token.  A lane takes words of four code bytes: weights 4g ..
// 4g + 3 and 4g + 16 .. 4g + 19 of a block.  q - 8 and d are exact in float32, so is
// their product; the scale rounds it once.  The row stays in registers for its
// norm.
//
// Bound by the bytes it writes: 8191 tokens of 2560 with a binary16 norm (126 MB out,
// 12 MB of the table) in 43 us.  A row's codes lie in pieces of 16 bytes, 256 bytes
// apart (the layout is the products'), so whole lines bring 76 MB
// where 12 are needed: 200 MB in all, 4.7 TB/s.  Five tokens take 4 us, one
// launch.  Non-temporal stores of h: 44.35 us a call, without 44.4.
#include "q4_0_device.h"
#include "q4_0_internal.h"

namespace q4 {

namespace {

typedef _Float16 h4_t __attribute__((ext_vector_type(4)));

constexpr int kMaxThreads = 1024;

template <bool YF16, int CH>
__global__ __launch_bounds__(kMaxThreads) void embed_kernel(EmbedArgs a) {
    __shared__ float sums[kMaxThreads / 64];
    const Layout L(a.vocab, a.in);
    const int words = (int)(a.in / 8);
    const int64_t t = blockIdx.x;
    const int token = a.tokens[t];
    const bool held = token >= 0 && token < a.vocab;
    const int64_t tile = held ? token / kTileRows : 0;
    const int r = held ? token % kTileRows : 0;
    const uint8_t *packed = (const uint8_t *)a.packed;
    uint32_t code[CH], d[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int w = threadIdx.x + i * blockDim.x;
        code[i] = 0x88888888u, d[i] = 0;
        if (held && w < words) {
            code[i] = load_u32(packed + L.code_off(tile, r, w & 3, w >> 2));
            d[i] = load_u16(packed + L.scale_off(tile, r, w >> 2));
        }
    }
    f4_t x[CH][2];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int w = threadIdx.x + i * blockDim.x;
        const float s = half_bits_to_float(d[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[i][0][e] = a.scale * (s * (float)((int)(code[i] >> (8 * e) & 15u) - 8));
            x[i][1][e] = a.scale * (s * (float)((int)(code[i] >> (8 * e + 4) & 15u) - 8));
            ss += x[i][0][e] * x[i][0][e] + x[i][1][e] * x[i][1][e];
        }
        if (w < words) {
            float *h = a.h + t * a.in + (w >> 2) * 32 + (w & 3) * 4;
            *(f4_t *)h = x[i][0];
            *(f4_t *)(h + 16) = x[i][1];
        }
    }
    if (!a.pre) return;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) ss += __shfl_xor(ss, m);
    const int waves = (blockDim.x + 63) / 64;
    if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int i = 0; i < waves; ++i) ss += sums[i];
    const float norm = 1.0f / sqrtf(ss / (float)a.in + a.eps);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int w = threadIdx.x + i * blockDim.x;
        if (w >= words) continue;
        const int at = (w >> 2) * 32 + (w & 3) * 4;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const float *pre = a.pre + at + 16 * p;
            f4_t y;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = x[i][p][e] * norm * (pre[e] + a.weight_offset);
            const int64_t o = t * a.in + at + 16 * p;
            if (YF16)
                *(h4_t *)((_Float16 *)a.y + o) =
                    h4_t{(_Float16)y[0], (_Float16)y[1], (_Float16)y[2], (_Float16)y[3]};
            else
                *(f4_t *)((float *)a.y + o) = y;
        }
    }
}

template <bool YF16, int CH> hipError_t launch(const EmbedArgs &a, hipStream_t stream) {
    const int64_t words = a.in / 8;
    const int64_t threads = ((words + CH - 1) / CH + 63) / 64 * 64;
    hipLaunchKernelGGL((embed_kernel<YF16, CH>), dim3((uint32_t)a.n), dim3((uint32_t)threads), 0,
                       stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_embed(const EmbedArgs &a, int y_f16, hipStream_t stream) {
    if (a.in <= 2 * 8 * kMaxThreads)
        return y_f16 ? launch<true, 2>(a, stream) : launch<false, 2>(a, stream);
    return y_f16 ? launch<true, 4>(a, stream) : launch<false, 4>(a, stream);
}

}  // namespace q4
