// latent_attention.cu -- absorbed latent attention over the paged cache
// (paged_latent_attention): one CTA per (query token, 8 heads), a warp a head,
// cache rows staged 16 tokens at a time, online softmax in fp32.
#include <cuda_fp16.h>

#include <cmath>

#include "pagedkv_latent.h"
#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "rope_latent.h"

namespace pkv {
namespace {

constexpr int kWarps = 8;
constexpr int kTile = 16;

template <int R, int P>
__global__ void __launch_bounds__(32 * kWarps) latent_attention_kernel(const LatentAttentionArgs a) {
    constexpr int E = R + P, N = E / 64, NV = R / 64;  // half2 pieces a lane holds
    __shared__ __align__(16) __half2 tile[kTile][E / 2];
    __shared__ long long rows[kTile];
    const int i = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x * kWarps + warp;
    int b = i, n = 1, first = i;
    if (a.query_start) {
        int lo = 0, hi = a.num_seqs;
        if (i < a.query_start[0] || i >= a.query_start[a.num_seqs]) return;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (a.query_start[mid] <= i) lo = mid; else hi = mid;
        }
        b = lo;
        first = a.query_start[b];
        n = a.query_start[b + 1] - first;
    }
    const int L = a.context_lens[b];
    const bool empty = !a.query_start && L == 0;
    if (L < 0 || L > a.max_context_len || n > a.max_q_len || (n > L && !empty)) {
        if (threadIdx.x == 0) flag_error(a.err, PKV_ERRBIT_CONTEXT);
        return;
    }
    const int end = empty ? 0 : L - n + (i - first) + 1;  // tokens this row attends
    float2 q[N], o[NV];
    const __half2 *qp = static_cast<const __half2 *>(a.q) +
                        (static_cast<long long>(i) * a.n_q_heads + (h < a.n_q_heads ? h : 0)) * (E / 2);
#pragma unroll
    for (int c = 0; c < N; ++c) q[c] = __half22float2(qp[lane + 32 * c]);
#pragma unroll
    for (int c = 0; c < NV; ++c) o[c] = make_float2(0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    for (int t0 = 0; t0 < end; t0 += kTile) {
        __syncthreads();
        if (threadIdx.x < kTile) {
            const int t = t0 + threadIdx.x;
            long long row = -1;
            if (t < end) {
                const int id = a.block_tables[static_cast<long long>(b) * a.max_blocks_per_seq +
                                              t / a.block_size];
                if (id < 0 || id >= a.num_blocks)
                    flag_error(a.err, PKV_ERRBIT_BLOCK_ID);
                else
                    row = static_cast<long long>(id) * a.block_size + t % a.block_size;
            }
            rows[threadIdx.x] = row;
        }
        __syncthreads();
        for (int x = threadIdx.x; x < kTile * (E / 8); x += 32 * kWarps) {
            const int r = x / (E / 8), c = x % (E / 8);
            if (rows[r] >= 0)
                reinterpret_cast<uint4 *>(tile[r])[c] =
                    static_cast<const uint4 *>(a.cache)[rows[r] * (E / 8) + c];
        }
        __syncthreads();
        for (int r = 0; r < kTile; ++r) {
            if (rows[r] < 0) continue;
            float s = 0.f;
            float2 k[N];
#pragma unroll
            for (int c = 0; c < N; ++c) {
                k[c] = __half22float2(tile[r][lane + 32 * c]);
                s += q[c].x * k[c].x + q[c].y * k[c].y;
            }
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            s *= a.negate ? -a.scale_log2 : a.scale_log2;
            const float mn = fmaxf(m, s);
            const float f = exp2f(m - mn), p = exp2f(s - mn);
            m = mn;
            l = l * f + p;
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                o[c].x = o[c].x * f + p * k[c].x;
                o[c].y = o[c].y * f + p * k[c].y;
            }
        }
    }
    if (h >= a.n_q_heads) return;
    const long long row = static_cast<long long>(i) * a.n_q_heads + h;
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int c = 0; c < NV; ++c)
        static_cast<__half2 *>(a.out)[row * (R / 2) + lane + 32 * c] =
            __floats2half2_rn(o[c].x * inv, o[c].y * inv);
    if (a.lse_out && lane == 0)
        a.lse_out[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

cudaError_t launch_latent_attention(const LatentAttentionArgs &a, cudaStream_t stream) {
    if (a.total_q > 65535) return cudaErrorInvalidValue;
    const dim3 grid((a.n_q_heads + kWarps - 1) / kWarps, a.total_q);
    if (a.latent_dim == 512)
        latent_attention_kernel<512, 64><<<grid, 32 * kWarps, 0, stream>>>(a);
    else
        latent_attention_kernel<256, 64><<<grid, 32 * kWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pkv
