// latent_prefill.cu -- expanded latent attention of prompts
// (latent_prefill_attention): one warp per (query, head), online softmax.
#include <cuda_fp16.h>

#include <cmath>

#include "pagedkv_latent.h"
#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "rope_latent.h"

namespace pkv {
namespace {

constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) latent_prefill_kernel(const LatentPrefillArgs a) {
    constexpr int P = 64, N = D / 64;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y;
    const int i = blockIdx.x * kWarps + warp;
    if (i >= a.total_q || i < a.q_start[0] || i >= a.q_start[a.num_seqs]) return;
    int lo = 0, hi = a.num_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.q_start[mid] <= i) lo = mid; else hi = mid;
    }
    const int q0 = a.q_start[lo], n = a.q_start[lo + 1] - q0;
    const int k0 = a.kv_start[lo], m_b = a.kv_start[lo + 1] - k0;
    if (n > m_b || n > a.max_q_len || m_b > a.max_kv_len || k0 < 0 || k0 + m_b > a.total_kv) {
        if (lane == 0) flag_error(a.err, PKV_ERRBIT_CONTEXT);
        return;
    }
    const int end = m_b - n + (i - q0) + 1;
    const long long row = static_cast<long long>(i) * a.n_heads + h;
    const __half2 *qp = static_cast<const __half2 *>(a.q) + row * ((D + P) / 2);
    float2 q[N + 1], o[N];
#pragma unroll
    for (int c = 0; c <= N; ++c) q[c] = __half22float2(qp[lane + 32 * c]);
#pragma unroll
    for (int c = 0; c < N; ++c) o[c] = make_float2(0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    for (int t = 0; t < end; ++t) {
        const __half2 *kp = static_cast<const __half2 *>(a.kv) +
                            (static_cast<long long>(k0 + t) * a.n_heads + h) * D;
        const float2 r = __half22float2(
            (static_cast<const __half2 *>(a.k_rope) + static_cast<long long>(k0 + t) * (P / 2))[lane]);
        float s = q[N].x * r.x + q[N].y * r.y;
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const float2 k = __half22float2(kp[lane + 32 * c]);
            s += q[c].x * k.x + q[c].y * k.y;
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.scale_log2;
        const float mn = fmaxf(m, s);
        const float f = exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const float2 v = __half22float2(kp[D / 2 + lane + 32 * c]);
            o[c].x = o[c].x * f + p * v.x;
            o[c].y = o[c].y * f + p * v.y;
        }
    }
    const float inv = 1.f / l;
#pragma unroll
    for (int c = 0; c < N; ++c)
        static_cast<__half2 *>(a.out)[row * (D / 2) + lane + 32 * c] =
            __floats2half2_rn(o[c].x * inv, o[c].y * inv);
    if (a.lse_out && lane == 0) a.lse_out[row] = (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, cudaStream_t stream) {
    const dim3 grid((a.total_q + kWarps - 1) / kWarps, a.n_heads);
    if (a.head_dim == 128)
        latent_prefill_kernel<128><<<grid, 32 * kWarps, 0, stream>>>(a);
    else
        latent_prefill_kernel<64><<<grid, 32 * kWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pkv
