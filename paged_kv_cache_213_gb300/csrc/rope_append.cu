// rope_append.cu -- RMS norm of query and key heads, rotation by position and
// the append into the paged cache in one pass: the per-head form
// (paged_qk_norm_rope_append, fp16 and E4M3 caches) and the latent form
// (paged_latent_append).  Formulas: include/pagedkv_rope.h.
//
// Both are bound by memory at prompt sizes and by the latency of one dependent
// chain (slot and position, then the rotation's row) at decode sizes.  A
// thread holds 8 consecutive entries of a head (one 16-byte load, one store),
// the d/8 threads of a head reduce its sum of squares by shuffles, and the
// partner of a split-half pair sits a fixed number of lanes away, so nothing
// goes through shared memory and every input byte is read once.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "e4m3_quant.cuh"
#include "pagedkv_rope.h"
#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "rope_latent.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
    return make_uint4(pack_half2(y[0], y[1]), pack_half2(y[2], y[3]), pack_half2(y[4], y[5]),
                      pack_half2(y[6], y[7]));
}

// 8 fp32 values to 8 E4M3 codes of y / scale (the rounding of quantize16).
__device__ __forceinline__ uint2 quantize8(const float (&y)[8], float scale) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __nv_fp8x2_storage_t a = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(y[4 * i], scale), __fdiv_rn(y[4 * i + 1], scale)),
            __NV_SATFINITE, __NV_E4M3);
        const __nv_fp8x2_storage_t b = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(y[4 * i + 2], scale), __fdiv_rn(y[4 * i + 3], scale)),
            __NV_SATFINITE, __NV_E4M3);
        w[i] = static_cast<uint32_t>(a) | (static_cast<uint32_t>(b) << 16);
    }
    return make_uint2(w[0], w[1]);
}

// Rotates the 8 entries y (entries 8 j .. 8 j + 7 of a vector) by the table row
// cs (cos, then sin, rot / 2 each).  Split halves: the partner entries are
// rot / 16 lanes up or down; every lane of the warp calls this.
__device__ __forceinline__ void rotate8(float (&y)[8], const float *cs, int j, int rot,
                                        bool interleaved, bool active) {
    const int half = rot / 2;
    if (interleaved) {
        if (!active || 8 * j >= rot) return;
        const float4 c = *reinterpret_cast<const float4 *>(cs + 4 * j);
        const float4 s = *reinterpret_cast<const float4 *>(cs + half + 4 * j);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = y[2 * i], b = y[2 * i + 1];
            y[2 * i] = a * cc[i] - b * ss[i];
            y[2 * i + 1] = b * cc[i] + a * ss[i];
        }
        return;
    }
    const int h8 = half / 8;
    const bool low = j < h8;
    const bool turned = j < 2 * h8;
    const int lane = threadIdx.x & 31;
    const int src = turned ? (low ? lane + h8 : lane - h8) : lane;
    float other[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = __shfl_sync(0xffffffffu, y[i], src);
    if (!active || !turned) return;
    const int p = 8 * (low ? j : j - h8);
    const float4 c0 = *reinterpret_cast<const float4 *>(cs + p);
    const float4 c1 = *reinterpret_cast<const float4 *>(cs + p + 4);
    const float4 s0 = *reinterpret_cast<const float4 *>(cs + half + p);
    const float4 s1 = *reinterpret_cast<const float4 *>(cs + half + p + 4);
    const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        // low half: a cos - b sin; high half: b cos + a sin
        y[i] = low ? y[i] * cc[i] - other[i] * ss[i] : y[i] * cc[i] + other[i] * ss[i];
}

// The slot and the rotation row of a token; false for a token that is skipped
// (padding, or flagged once by the thread that has `tell`).
__device__ __forceinline__ bool token_place(const int64_t *slots, const int32_t *positions,
                                            long long num_slots, int max_positions, int rot,
                                            int token, bool tell, int32_t *err, long long *slot,
                                            int *position) {
    const long long s = slots[token];
    const int p = rot > 0 ? positions[token] : 0;
    *slot = s;
    *position = p;
    if (s < 0) return false;
    const bool bad_slot = s >= num_slots;
    const bool bad_pos = rot > 0 && (p < 0 || p >= max_positions);
    if (tell && bad_slot) flag_error(err, PKV_ERRBIT_SLOT);
    if (tell && bad_pos) flag_error(err, PKV_ERRBIT_POSITION);
    return !bad_slot && !bad_pos;
}

// One group of `width` lanes per (token, head); heads 0 .. H-1 are queries,
// then Hk keys, then Hk values.
template <bool F8>
__global__ void __launch_bounds__(kThreads) qk_append_kernel(const QkAppendArgs a) {
    allow_dependent_launch();  // the attention kernel may get scheduled meanwhile
    const int heads = a.n_q_heads + 2 * a.n_kv_heads;
    const unsigned unit = (blockIdx.x * kThreads + threadIdx.x) >> a.width_log2;
    const int j = threadIdx.x & ((1 << a.width_log2) - 1);
    const bool in_grid = unit < static_cast<unsigned>(a.num_tokens) * heads;
    const int token = in_grid ? unit / heads : 0;
    const int head = in_grid ? unit - token * heads : 0;
    const bool is_q = head < a.n_q_heads;
    const bool is_v = head >= a.n_q_heads + a.n_kv_heads;
    const int kv_head = head - a.n_q_heads - (is_v ? a.n_kv_heads : 0);
    const int d = a.head_dim;
    bool active = in_grid && 8 * j < d;
    const __half *x = static_cast<const __half *>(is_q ? a.q : is_v ? a.v : a.k) +
                      token * (is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride) +
                      (is_q ? head : kv_head) * d + 8 * j;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (active) raw = *reinterpret_cast<const uint4 *>(x);
    long long slot = -1;
    int position = 0;
    const bool keep = token_place(a.slot_mapping, a.positions, a.num_slots, a.max_positions,
                                  a.rot_dim, token, in_grid && head == 0 && j == 0, a.err, &slot,
                                  &position);
    active = active && keep;
    if (!keep) position = 0;  // a row that exists: the lanes below load nothing of it
    float y[8];
    unpack8(raw, y);
    const __half *w = static_cast<const __half *>(is_q ? a.q_weight : a.k_weight);
    // the whole warp runs the shuffles; values pass through untouched
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += y[i] * y[i];
    for (int o = (1 << a.width_log2) / 2; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (!is_v && w && active) {
        const float inv = 1.f / sqrtf(sum / static_cast<float>(d) + a.eps);
        float wf[8];
        unpack8(*reinterpret_cast<const uint4 *>(w + 8 * j), wf);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * inv * wf[i];
    }
    if (a.rot_dim > 0) {
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = y[i];
        rotate8(z, a.cos_sin + static_cast<long long>(position) * a.rot_dim, j, a.rot_dim,
                a.interleaved, active && !is_v);
        if (!is_v)
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = z[i];
    }
    if (!active) return;
    if (is_q) {
        __half *dst = static_cast<__half *>(a.q_out) +
                      (static_cast<long long>(token) * a.n_q_heads + head) * d + 8 * j;
        *reinterpret_cast<uint4 *>(dst) = pack8(y);
        return;
    }
    const long long block = slot / a.block_size;
    const long long row = slot - block * a.block_size;
    const long long dst = ((block * a.n_kv_heads + kv_head) * a.block_size + row) * d + 8 * j;
    if (F8) {
        unsigned char *cache = static_cast<unsigned char *>(is_v ? a.v_cache : a.k_cache);
        *reinterpret_cast<uint2 *>(cache + dst) = quantize8(y, is_v ? a.v_scale : a.k_scale);
    } else {
        __half *cache = static_cast<__half *>(is_v ? a.v_cache : a.k_cache);
        *reinterpret_cast<uint4 *>(cache + dst) = is_v ? raw : pack8(y);
    }
}

// One warp per job.  Job 0 of a token: its latent (32 lanes x 8 entries a
// step) and the rotated key part; job j > 0: query heads (j - 1) * kHeadSteps
// * (32 / width) and on, `width` lanes a head.
constexpr int kHeadSteps = 4;
constexpr int kMaxLatentSteps = 4;  // 1024 entries

__global__ void __launch_bounds__(kThreads) latent_append_kernel(const LatentAppendArgs a) {
    allow_dependent_launch();
    const unsigned job = (blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (job >= static_cast<unsigned>(a.num_tokens) * a.jobs) return;
    const int token = job / a.jobs;
    const int part = job - token * a.jobs;
    const int R = a.latent_dim, P = a.rope_dim;
    const int j = lane & ((1 << a.width_log2) - 1);
    if (part == 0) {
        const __half *x = static_cast<const __half *>(a.kv) + token * a.kv_stride;
        uint4 raw[kMaxLatentSteps];
#pragma unroll
        for (int i = 0; i < kMaxLatentSteps; ++i) {
            const int e = 8 * (lane + 32 * i);
            raw[i] = e < R ? *reinterpret_cast<const uint4 *>(x + e) : make_uint4(0, 0, 0, 0);
        }
        uint4 rope = make_uint4(0, 0, 0, 0);
        if (8 * lane < P) rope = *reinterpret_cast<const uint4 *>(x + R + 8 * lane);
        long long slot;
        int position;
        if (!token_place(a.slot_mapping, a.positions, a.num_slots, a.max_positions, P, token,
                         lane == 0, a.err, &slot, &position))
            return;
        __half *row = static_cast<__half *>(a.cache) + slot * (R + P);
        float y[8];
        unpack8(rope, y);
        rotate8(y, a.cos_sin + static_cast<long long>(position) * P, lane, P, a.interleaved,
                8 * lane < P);
        if (8 * lane < P) *reinterpret_cast<uint4 *>(row + R + 8 * lane) = pack8(y);
        const __half *w = static_cast<const __half *>(a.weight);
        if (!w) {
#pragma unroll
            for (int i = 0; i < kMaxLatentSteps; ++i) {
                const int e = 8 * (lane + 32 * i);
                if (e < R) *reinterpret_cast<uint4 *>(row + e) = raw[i];
            }
            return;
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kMaxLatentSteps; ++i) {
            unpack8(raw[i], y);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += y[k] * y[k];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = 1.f / sqrtf(sum / static_cast<float>(R) + a.eps);
#pragma unroll
        for (int i = 0; i < kMaxLatentSteps; ++i) {
            const int e = 8 * (lane + 32 * i);
            if (e < R) {
                float wf[8];
                unpack8(*reinterpret_cast<const uint4 *>(w + e), wf);
                unpack8(raw[i], y);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = y[k] * inv * wf[k];
                *reinterpret_cast<uint4 *>(row + e) = pack8(y);
            }
        }
        return;
    }
    const int per_step = 32 >> a.width_log2;
    const int first = (part - 1) * kHeadSteps * per_step + (lane >> a.width_log2);
    const __half *x = static_cast<const __half *>(a.q_rope) + token * a.q_token_stride + 8 * j;
    uint4 raw[kHeadSteps];
#pragma unroll
    for (int i = 0; i < kHeadSteps; ++i) {
        const int h = first + i * per_step;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (h < a.n_q_heads && 8 * j < P)
            raw[i] = *reinterpret_cast<const uint4 *>(x + h * a.q_head_stride);
    }
    long long slot;
    int position;
    if (!token_place(a.slot_mapping, a.positions, a.num_slots, a.max_positions, P, token, false,
                     nullptr, &slot, &position))
        return;
    __half *out = static_cast<__half *>(a.q_out) + token * a.out_token_stride + 8 * j;
#pragma unroll
    for (int i = 0; i < kHeadSteps; ++i) {
        const int h = first + i * per_step;
        const bool active = h < a.n_q_heads && 8 * j < P;
        float y[8];
        unpack8(raw[i], y);
        rotate8(y, a.cos_sin + static_cast<long long>(position) * P, j, P, a.interleaved, active);
        if (active) *reinterpret_cast<uint4 *>(out + h * a.out_head_stride) = pack8(y);
    }
}

int log2_lanes(int entries) {  // lanes of 8 entries, rounded up to a power of two
    int w = 0;
    while ((8 << w) < entries) ++w;
    return w;
}

}  // namespace

cudaError_t launch_qk_append(QkAppendArgs a, bool fp8, cudaStream_t stream) {
    a.width_log2 = log2_lanes(a.head_dim);
    const long long units =
        static_cast<long long>(a.num_tokens) * (a.n_q_heads + 2 * a.n_kv_heads);
    const long long blocks = ((units << a.width_log2) + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL || (units << a.width_log2) > 0xffffffffLL)
        return cudaErrorInvalidValue;
    if (fp8)
        qk_append_kernel<true><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
    else
        qk_append_kernel<false><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_latent_append(LatentAppendArgs a, cudaStream_t stream) {
    a.width_log2 = log2_lanes(a.rope_dim);
    const int per_job = kHeadSteps * (32 >> a.width_log2);
    a.jobs = 1 + (a.n_q_heads + per_job - 1) / per_job;
    const long long threads = static_cast<long long>(a.num_tokens) * a.jobs * 32;
    const long long blocks = (threads + kThreads - 1) / kThreads;
    if (threads > 0xffffffffLL) return cudaErrorInvalidValue;
    latent_append_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pkv
