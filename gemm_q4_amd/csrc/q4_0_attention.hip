// Attention of a ragged batch over the paged cache.
//
// The plainest kernel that is right for every case: one workgroup per token
// and query head, its four waves taking every fourth visible key, lanes across
// the head's elements, running maximum and sum of the softmax per wave, the
// four waves' results joined at the end.
#include "q4_0_device.h"
#include "q4_0_internal.h"

namespace q4 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <bool F16, int DIM>
__global__ __launch_bounds__(256) void attention_kernel(AttentionArgs a) {
    constexpr int PER = DIM / 64;
    __shared__ float acc_s[4][DIM];
    __shared__ float m_s[4], l_s[4];
    const int h = blockIdx.x % a.q_heads;
    const int t = blockIdx.x / a.q_heads;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    // the conversation that holds token t
    int s = -1, first = 0, last = 0;
    for (int i = 0; i < a.batch; ++i) {
        const int b = a.q_start[i], e = a.q_start[i + 1];
        if (t >= b && t < e) s = i, first = b, last = e;
    }
    if (s < 0) return;
    const int p = a.kv_len[s] - (last - first) + (t - first);
    const int heads = a.cache.heads, shift = a.cache.page_shift;
    const int hk = h / (a.q_heads / heads);
    float q[PER], acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t at = (int64_t)t * a.q_stride + h * DIM + i * 64 + lane;
        q[i] = F16 ? (float)((const _Float16 *)a.q)[at] : ((const float *)a.q)[at];
        acc[i] = 0.0f;
    }
    const int lo = a.window && p >= a.window ? p - a.window + 1 : 0;
    float m = -INFINITY, l = 0.0f;
    bool bad = false;
    for (int j = wave; j <= p; j += 4) {
        if (j < lo && j >= a.sinks) {
            j += (lo - j) / 4 * 4;
            if (j < lo) continue;
        }
        const int slot = j >> shift;
        const int page = slot < a.table_stride ? a.table[(int64_t)s * a.table_stride + slot] : -1;
        if (page < 0 || page >= a.cache.pages) {
            bad = true;
            continue;
        }
        const int64_t row =
            ((((int64_t)page * heads + hk) << shift) + (j & ((1 << shift) - 1))) * DIM;
        float d = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) d += q[i] * (float)a.cache.k[row + i * 64 + lane];
#pragma unroll
        for (int x = 32; x > 0; x >>= 1) d += __shfl_xor(d, x);
        d *= a.scale * kLog2e;
        const float mn = fmaxf(m, d);
        const float f = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
        const float w = __builtin_amdgcn_exp2f(d - mn);
        m = mn;
        l = l * f + w;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            acc[i] = acc[i] * f + w * (float)a.cache.v[row + i * 64 + lane];
    }
    if (bad) l = NAN;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc_s[wave][i * 64 + lane] = acc[i];
    if (lane == 0) m_s[wave] = m, l_s[wave] = l;
    __syncthreads();
    float mm = -INFINITY;
    for (int w = 0; w < 4; ++w) mm = fmaxf(mm, m_s[w]);
    float ll = 0.0f, f[4];
    for (int w = 0; w < 4; ++w) {
        f[w] = m_s[w] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m_s[w] - mm);
        ll += l_s[w] == l_s[w] ? l_s[w] * f[w] : l_s[w];
    }
    for (int i = threadIdx.x; i < DIM; i += 256) {
        float y = 0.0f;
        for (int w = 0; w < 4; ++w)
            if (f[w] != 0.0f) y += acc_s[w][i] * f[w];
        y = p < 0 ? 0.0f : y / ll;
        const int64_t at = ((int64_t)t * a.q_heads + h) * DIM + i;
        if (F16)
            ((_Float16 *)a.y)[at] = (_Float16)y;
        else
            ((float *)a.y)[at] = y;
    }
}

template <bool F16> hipError_t by_dim(const AttentionArgs &a, hipStream_t stream) {
    const dim3 grid((uint32_t)a.n * (uint32_t)a.q_heads);
    if (a.cache.dim == 64)
        hipLaunchKernelGGL((attention_kernel<F16, 64>), grid, dim3(256), 0, stream, a);
    else if (a.cache.dim == 128)
        hipLaunchKernelGGL((attention_kernel<F16, 128>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((attention_kernel<F16, 256>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

bool attention_supports(int dim) { return dim == 64 || dim == 128 || dim == 256; }

size_t attention_workspace_bytes(const AttentionArgs &, int) { return 0; }

hipError_t launch_attention(const AttentionArgs &a, int x_f16, void *, hipStream_t stream) {
    return x_f16 ? by_dim<true>(a, stream) : by_dim<false>(a, stream);
}

}  // namespace q4
