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
// goes through shared memory and every input byte is read once.  8191 tokens x 80
// heads of 128 into E4M3: 60 us, 5.4 TB/s (79 % of the copy rate); 8003 tokens x 128
// query heads, latent: 47 us, 6.0 TB/s; up to some 64 tokens 2.4 us.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "f32x2.cuh"
#include "pagedkv_rope.h"
#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "rope_latent.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;  // 256: 62 -> 65 us (the 8191-token case below), 47.0 -> 47.8 (latent)

__device__ __forceinline__ uint4 pack8(const float2 (&y)[4]) {
    return make_uint4(pack_half2(y[0].x, y[0].y), pack_half2(y[1].x, y[1].y),
                      pack_half2(y[2].x, y[2].y), pack_half2(y[3].x, y[3].y));
}

__device__ __forceinline__ void unpack8(const uint4 &v, float2 (&f)[4]) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __half22float2(h[i]);
}

// 8 fp32 values to 8 E4M3 codes of y / scale, to the codes that paged_kv_append_fp8
// stores.  inv = RN(1 / scale), or 0 for a scale that divide2 does not take.
__device__ __forceinline__ uint2 quantize8(const float2 (&y)[4], float scale, float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 q;
        if (inv != 0.f)
            q = divide2(y[i], scale, inv);
        else
            q = make_float2(__fdiv_rn(y[i].x, scale), __fdiv_rn(y[i].y, scale));
        w[i] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The cosines and sines that entries 8 j .. 8 j + 7 of a vector need, from the
// table row cs (cos, then sin, rot / 2 each): 8 pairs of split halves, or 4
// interleaved ones.  Beyond rot: cos 1, sin 0.
struct Turn {
    float c[8], s[8];
};

__device__ __forceinline__ void load4(float *d, const float *p) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    d[0] = v.x;
    d[1] = v.y;
    d[2] = v.z;
    d[3] = v.w;
}

__device__ __forceinline__ Turn load_turn(const float *cs, int j, int rot, bool interleaved) {
    Turn t;
#pragma unroll
    for (int i = 0; i < 8; ++i) t.c[i] = 1.f, t.s[i] = 0.f;
    if (8 * j >= rot) return t;
    const int half = rot / 2;
    if (interleaved) {
        load4(t.c, cs + 4 * j);
        load4(t.s, cs + half + 4 * j);
    } else {
        const bool low = 8 * j < half;
        const int p = low ? 8 * j : 8 * j - half;
        load4(t.c, cs + p);
        load4(t.c + 4, cs + p + 4);
        load4(t.s, cs + half + p);
        load4(t.s + 4, cs + half + p + 4);
        // low half: a cos - b sin; high half: b cos + a sin
#pragma unroll
        for (int i = 0; i < 8; ++i) t.s[i] = low ? -t.s[i] : t.s[i];
    }
    return t;
}

// Rotates the 8 entries y (entries 8 j .. of a vector) by t; those beyond rot stay bit
// for bit (cos 1 and sin 0 would make NaN of an infinity and 0 of -0).  Split halves:
// the partner entries are rot / 16 lanes up or down; every lane of the warp calls this.
__device__ __forceinline__ void rotate8(float2 (&y)[4], const Turn &t, int j, int rot,
                                        bool interleaved) {
    const bool turns = 8 * j < rot;
    if (interleaved) {
        if (!turns) return;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // (a cos - b sin, b cos + a sin)
            y[i] = fma2(y[i], make_float2(t.c[i], t.c[i]),
                        mul2(make_float2(y[i].y, y[i].x), make_float2(-t.s[i], t.s[i])));
        return;
    }
    const int h8 = rot / 16;
    const int lane = threadIdx.x & 31;
    const int src = j < h8 ? lane + h8 : j < 2 * h8 ? lane - h8 : lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 other = make_float2(__shfl_sync(0xffffffffu, y[i].x, src),
                                         __shfl_sync(0xffffffffu, y[i].y, src));
        if (turns)
            y[i] = fma2(other, make_float2(t.s[2 * i], t.s[2 * i + 1]),
                        mul2(y[i], make_float2(t.c[2 * i], t.c[2 * i + 1])));
    }
}

// y * inv * w, and the sum of squares.
__device__ __forceinline__ void scale8(float2 (&y)[4], float inv, const float2 (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul2(mul2(y[i], make_float2(inv, inv)), w[i]);
}
__device__ __forceinline__ float squares8(const float2 (&y)[4]) {
    float2 s = mul2(y[0], y[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s = fma2(y[i], y[i], s);
    return s.x + s.y;
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

// One warp per job: U steps of 32 / width heads of a token and of one kind,
// `width` lanes a head, whose loads are all in flight together and which share the
// token's slot, rotation row and norm weights.  A token's first jobs take its
// queries, the next its keys, the others its values, which only move.
//  U = 4 where the warps fill the GPU anyway: with one head a lane too few bytes are
// in flight behind the chain from position to rotation row.  U = 1 for fewer: more
// warps, a shorter chain.
//  D = 64 or 128 knows the head size: with sizes of the call and heads of all kinds
// in a warp the kernel was bound by instruction issue (945 a warp; 8191 tokens x 80
// heads into E4M3 took 108 us).  D = 0 is any other size.
template <bool F8, int U, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) qk_append_kernel(const QkAppendArgs a) {
    grid_dependency_wait();
    allow_dependent_launch();  // the attention kernel may get scheduled meanwhile
    const int width = D > 0 ? D / 8 : 1 << a.width_log2;
    const int lane = threadIdx.x & 31, j = lane & (width - 1);
    const int per = 32 / width;  // heads of a step
    const unsigned job = (blockIdx.x * kThreads + threadIdx.x) >> 5;
    const unsigned token = job / a.jobs;
    if (token >= static_cast<unsigned>(a.num_tokens)) return;
    int part = job - token * a.jobs;
    const bool tell = part == 0 && lane == 0;
    const int H = a.n_q_heads, Hk = a.n_kv_heads, d = D > 0 ? D : a.head_dim;
    const bool inside = D > 0 || 8 * j < d;
    // the kind of the job's heads
    const bool is_q = part < a.q_jobs;
    part -= is_q ? 0 : a.q_jobs;
    const bool is_v = !is_q && part >= a.kv_jobs;
    part -= is_v ? a.kv_jobs : 0;
    const int heads = is_q ? H : Hk;
    const int first = part * per * U + lane / width;
    const __half *x = static_cast<const __half *>(is_q ? a.q : is_v ? a.v : a.k) +
                      token * (is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride) + first * d + 8 * j;
    // what is read once and what the attention reads much later pass L2 by (60 us; 62
    // with the default policies); the cache rows do not
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        raw[u] = make_uint4(0, 0, 0, 0);
        if (inside && first + u * per < heads)
            raw[u] = __ldcs(reinterpret_cast<const uint4 *>(x + u * per * d));
    }
    long long slot;
    int position;
    if (!token_place(a.slot_mapping, a.positions, a.num_slots, a.max_positions, a.rot_dim, token,
                     tell, a.err, &slot, &position))
        return;
    // 32-bit division where it will do: the 64-bit one is some 70 instructions
    const long long block = slot >> 32 ? slot / a.block_size
                                       : static_cast<unsigned>(slot) / static_cast<unsigned>(a.block_size);
    const long long row = slot - block * a.block_size;
    // where the first head goes (in entries), and a head further
    const long long dst =
        is_q ? (static_cast<long long>(token) * H + first) * d + 8 * j
             : ((block * Hk + first) * a.block_size + row) * d + 8 * j;
    const long long step = static_cast<long long>(per * d) * (is_q ? 1 : a.block_size);
    unsigned char *cache = static_cast<unsigned char *>(is_v ? a.v_cache : a.k_cache);
    if (is_v) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!inside || first + u * per >= heads) continue;
            const long long at = dst + u * step;
            if (F8) {
                float2 y[4];
                unpack8(raw[u], y);
                *reinterpret_cast<uint2 *>(cache + at) = quantize8(y, a.v_scale, a.v_inv);
            } else {
                *reinterpret_cast<uint4 *>(cache + 2 * at) = raw[u];
            }
        }
        return;
    }
    const bool turns = a.rot_dim > 0;
    Turn turn{};
    if (turns)
        turn = load_turn(a.cos_sin + static_cast<long long>(position) * a.rot_dim, j, a.rot_dim,
                         INTERLEAVED);
    const __half *w = static_cast<const __half *>(is_q ? a.q_weight : a.k_weight);
    float2 wf[4];
    if (w && inside) unpack8(*reinterpret_cast<const uint4 *>(w + 8 * j), wf);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float2 y[4];
        unpack8(raw[u], y);
        if (w) {
            float sum = squares8(y);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                if (o < width) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            scale8(y, rsqrtf(fmaf(sum, a.inv_dim, a.eps)), wf);
        }
        if (turns) rotate8(y, turn, j, a.rot_dim, INTERLEAVED);
        if (!inside || first + u * per >= heads) continue;
        const long long at = dst + u * step;
        if (is_q)
            __stcs(reinterpret_cast<uint4 *>(static_cast<__half *>(a.q_out) + at), pack8(y));
        else if (F8)
            *reinterpret_cast<uint2 *>(cache + at) = quantize8(y, a.k_scale, a.k_inv);
        else
            *reinterpret_cast<uint4 *>(cache + 2 * at) = pack8(y);
    }
}

// One warp per job.  Job 0 of a token: its latent (32 lanes x 8 entries a
// step) and the rotated key part; job j > 0: query heads (j - 1) * kHeadSteps
// * (32 / width) and on, `width` lanes a head.
constexpr int kHeadSteps = 8;  // 8003 tokens x 128 heads: 2 steps 62 us, 4 50.6, 8 47.8
constexpr int kMaxLatentSteps = 4;  // 1024 entries

__global__ void __launch_bounds__(kThreads) latent_append_kernel(const LatentAppendArgs a) {
    grid_dependency_wait();
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
        float2 y[4];
        unpack8(rope, y);
        rotate8(y, load_turn(a.cos_sin + static_cast<long long>(position) * P, lane, P,
                             a.interleaved), lane, P, a.interleaved);
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
            sum += squares8(y);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = rsqrtf(fmaf(sum, 1.f / static_cast<float>(R), a.eps));
#pragma unroll
        for (int i = 0; i < kMaxLatentSteps; ++i) {
            const int e = 8 * (lane + 32 * i);
            if (e < R) {
                float2 wf[4];
                unpack8(*reinterpret_cast<const uint4 *>(w + e), wf);
                unpack8(raw[i], y);
                scale8(y, inv, wf);
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
    const Turn turn =
        load_turn(a.cos_sin + static_cast<long long>(position) * P, j, P, a.interleaved);
    __half *out = static_cast<__half *>(a.q_out) + token * a.out_token_stride + 8 * j;
#pragma unroll
    for (int i = 0; i < kHeadSteps; ++i) {
        const int h = first + i * per_step;
        const bool active = h < a.n_q_heads && 8 * j < P;
        float2 y[4];
        unpack8(raw[i], y);
        rotate8(y, turn, j, P, a.interleaved);
        if (active) *reinterpret_cast<uint4 *>(out + h * a.out_head_stride) = pack8(y);
    }
}

int log2_lanes(int entries) {  // lanes of 8 entries, rounded up to a power of two
    int w = 0;
    while ((8 << w) < entries) ++w;
    return w;
}

}  // namespace

namespace {

template <bool F8, int U, int D>
cudaError_t launch_qk(QkAppendArgs a, cudaStream_t stream) {
    const int per_job = U * (32 >> a.width_log2);
    a.q_jobs = (a.n_q_heads + per_job - 1) / per_job;
    a.kv_jobs = (a.n_kv_heads + per_job - 1) / per_job;
    a.jobs = a.q_jobs + 2 * a.kv_jobs;
    a.inv_dim = 1.f / static_cast<float>(a.head_dim);
    auto inverse = [](float s) { return s >= 0x1p-60f && s <= 0x1p60f ? 1.f / s : 0.f; };
    a.k_inv = inverse(a.k_scale);
    a.v_inv = inverse(a.v_scale);
    const long long threads = static_cast<long long>(a.num_tokens) * a.jobs * 32;
    if (threads > 0xffffffffLL - kThreads) return cudaErrorInvalidValue;
    const unsigned blocks = static_cast<unsigned>((threads + kThreads - 1) / kThreads);
    return launch_pdl(a.interleaved ? qk_append_kernel<F8, U, D, true> : qk_append_kernel<F8, U, D, false>,
                      dim3(blocks), dim3(kThreads), 0, stream, a);
}

template <bool F8, int U>
cudaError_t launch_qk_sized(const QkAppendArgs &a, cudaStream_t stream) {
    return a.head_dim == 128  ? launch_qk<F8, U, 128>(a, stream)
           : a.head_dim == 64 ? launch_qk<F8, U, 64>(a, stream)
                              : launch_qk<F8, U, 0>(a, stream);
}

}  // namespace

cudaError_t launch_qk_append(QkAppendArgs a, bool fp8, cudaStream_t stream) {
    a.width_log2 = log2_lanes(a.head_dim);
    const long long lanes =
        (static_cast<long long>(a.num_tokens) * (a.n_q_heads + 2 * a.n_kv_heads)) << a.width_log2;
    // twice the threads that the GPU holds at once
    if (lanes > 600000)
        return fp8 ? launch_qk_sized<true, 4>(a, stream) : launch_qk_sized<false, 4>(a, stream);
    return fp8 ? launch_qk_sized<true, 1>(a, stream) : launch_qk_sized<false, 1>(a, stream);
}

cudaError_t launch_latent_append(LatentAppendArgs a, cudaStream_t stream) {
    a.width_log2 = log2_lanes(a.rope_dim);
    const int per_job = kHeadSteps * (32 >> a.width_log2);
    a.jobs = 1 + (a.n_q_heads + per_job - 1) / per_job;
    const long long threads = static_cast<long long>(a.num_tokens) * a.jobs * 32;
    const long long blocks = (threads + kThreads - 1) / kThreads;
    if (threads > 0xffffffffLL - kThreads) return cudaErrorInvalidValue;
    return launch_pdl(latent_append_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, a);
}

}  // namespace pkv
