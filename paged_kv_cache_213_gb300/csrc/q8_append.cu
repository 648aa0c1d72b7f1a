// q8_append.cu -- the append, the read-back and the block copy of the 8-bit
// caches with block scales (include/pagedkv_q8.h).
//
// Append.  The scale of a (block, head) needs the largest entry of all its new
// rows before the first code can be written, so whoever writes a block has all
// of them: a team of lanes holds the rows in registers, reduces their largest
// entry, and writes the codes from the same registers: one pass over memory.
// A token alone (decode) is a team of one row's lanes.
#include <cuda_fp16.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "q8.h"
#include "q8_codes.cuh"

namespace pkv {
namespace {

// Entries of the head that one lane takes: 16 bytes of fp16, 8 of codes.
constexpr int kPiece = 8;

// Largest finite |x| of 8 values.
__device__ __forceinline__ float top_of(const uint4 &x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
        if (lo < 0x7c00u) m = max(m, lo);
        if (hi < 0x7c00u) m = max(m, hi);
    }
    return __half2float(__ushort_as_half(static_cast<unsigned short>(m)));
}

// The scale after new tokens of largest entry `top`, and by how many powers of two
// it outgrew `had` (0: the block held nothing, or nothing but zeros).
template <int KIND>
__device__ __forceinline__ float grown(float had, float top, int *power) {
    *power = 0;
    if (!(had > 0.f)) return __fdiv_rn(top, q8_limit<KIND>());
    const float r = __fdiv_rn(top, __fmul_rn(had, q8_limit<KIND>()));
    if (!(r > 1.f)) return had;
    // r = (1 + f) 2^e: e + 1 unless f = 0
    const uint32_t bits = __float_as_uint(r);
    const int k = static_cast<int>(bits >> 23) - 127 + ((bits & 0x7fffffu) ? 1 : 0);
    *power = k;
    return ldexpf(had, k);
}

template <int KIND>
__device__ __forceinline__ uint2 quantised(const uint4 &x, float scale) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&x);
    const float s = scale > 0.f ? scale : 1.f;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        w[i] = q8_encode2<KIND>(__fdiv_rn(f.x, s), __fdiv_rn(f.y, s));
    }
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Codes of earlier tokens, whose scale grew by 2^power: code * 2^-power.
template <int KIND>
__device__ __forceinline__ uint2 shrunk(const uint2 &c, int power) {
    const float f = ldexpf(1.f, -power);
    const uint32_t w[2] = {c.x, c.y};
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = q8_widen<KIND, 0>(w[i]), hi = q8_widen<KIND, 1>(w[i]);
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        r[i] = q8_encode2<KIND>(a.x * f, a.y * f) | (q8_encode2<KIND>(b.x * f, b.y * f) << 16);
    }
    return make_uint2(r[0], r[1]);
}

// One token a sequence: a team of D / 8 lanes for each (sequence, head, K or V).
template <int KIND, int D>
__global__ void __launch_bounds__(128) q8_append_one_kernel(const Q8AppendArgs a) {
    constexpr int kTeam = D / kPiece;
    grid_dependency_wait();
    allow_dependent_launch();
    const long long team = (static_cast<long long>(blockIdx.x) * 128 + threadIdx.x) / kTeam;
    const int lane = threadIdx.x % kTeam;
    const int side = static_cast<int>(team & 1);
    const long long pair = team >> 1;
    const int b = static_cast<int>(pair / a.n_kv_heads), h = static_cast<int>(pair % a.n_kv_heads);
    // no thread leaves before the shuffles: a warp holds several teams
    bool live = b < a.num_seqs;
    int token = b, len = 0;
    if (live) {
        len = a.context_lens[b];
        int n = 1;
        if (a.query_start) {
            token = a.query_start[b];
            n = a.query_start[b + 1] - token;
        } else if (len == 0) {
            n = 0;
        }
        const bool ok = n >= 0 && n <= 1 && n <= len && token >= 0 && token + n <= a.total &&
                        len <= static_cast<long long>(a.max_blocks_per_seq) * a.block_size;
        if (!ok && lane == 0 && h == 0 && side == 0) flag_error(a.err, PKV_ERRBIT_CONTEXT);
        live = ok && n == 1;
    }
    uint4 x = make_uint4(0, 0, 0, 0);
    long long block = -1;
    int row = 0;
    if (live) {
        const uint4 *src = static_cast<const uint4 *>(side ? a.v_new : a.k_new);
        x = __ldcs(src + (token * (side ? a.v_stride : a.k_stride) + h * D) / kPiece + lane);
        const int j = (len - 1) / a.block_size;
        row = (len - 1) - j * a.block_size;
        block = a.block_tables[static_cast<long long>(b) * a.max_blocks_per_seq + j];
        if (block < 0 || block >= a.num_blocks) {
            if (lane == 0 && h == 0 && side == 0) flag_error(a.err, PKV_ERRBIT_BLOCK_ID);
            live = false;
        }
    }
    float top = top_of(x);
#pragma unroll
    for (int d = kTeam / 2; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    if (!live) return;
    const long long cell = block * a.n_kv_heads + h;
    float *scales = side ? a.v_scales : a.k_scales;
    const float had = row > 0 ? scales[cell] : 0.f;
    int power;
    const float scale = grown<KIND>(had, top, &power);
    uint2 *rows = static_cast<uint2 *>(side ? a.v_cache : a.k_cache) + cell * a.block_size * kTeam + lane;
    rows[row * kTeam] = quantised<KIND>(x, scale);
    if (power > 0)
        for (int r = 0; r < row; ++r) rows[r * kTeam] = shrunk<KIND>(rows[r * kTeam], power);
    if (lane == 0 && (row == 0 || scale != had)) scales[cell] = scale;
}

// Several tokens a sequence.  A CTA takes one block that a sequence touches and
// 128 / block_size heads of it (one head from 128 rows on), eight warps of 16 rows
// each (32 at 256 rows a block); the warps of a head exchange their largest entries.
//
// Which block: the blocks of sequence b get the numbers from start[b] / bs + 2 b on.
// A run of n tokens touches at most n / bs + 2 blocks (rounded down), so the ranges do
// not meet, and a CTA finds its sequence without a sum over the ones before.
constexpr int kWarps = 8;

template <int KIND, int D, int ROWS>  // rows of a warp
__global__ void __launch_bounds__(kWarps * 32) q8_append_many_kernel(const Q8AppendArgs a) {
    constexpr int kTeam = D / kPiece;        // lanes of a row
    constexpr int kAt = 32 / kTeam;          // rows of one load
    constexpr int kSteps = ROWS / kAt;
    grid_dependency_wait();
    allow_dependent_launch();
    __shared__ int which;
    __shared__ float tops[2][kWarps];
    const long long v = blockIdx.x;
    const int bs = a.block_size;
    if (threadIdx.x == 0) which = -1;
    __syncthreads();
    for (int b = threadIdx.x; b < a.num_seqs; b += kWarps * 32) {
        const int s = a.query_start[b], e = a.query_start[b + 1];
        if (s < 0 || e < s || e > a.total) {
            if (v == 0 && blockIdx.y == 0) flag_error(a.err, PKV_ERRBIT_CONTEXT);
            continue;
        }
        if (s / bs + 2ll * b <= v && v < e / bs + 2ll * (b + 1)) which = b;
    }
    __syncthreads();
    const int b = which;
    if (b < 0) return;
    const int s = a.query_start[b], n = a.query_start[b + 1] - s, len = a.context_lens[b];
    const int slot = static_cast<int>(v - (s / bs + 2ll * b));
    if (n > a.max_q_len || n > len ||
        len > static_cast<long long>(a.max_blocks_per_seq) * bs) {
        if (threadIdx.x == 0 && slot == 0 && blockIdx.y == 0) flag_error(a.err, PKV_ERRBIT_CONTEXT);
        return;
    }
    const int first = len - n, j = first / bs + slot;
    if (n == 0 || static_cast<long long>(j) * bs >= len) return;
    const long long block = a.block_tables[static_cast<long long>(b) * a.max_blocks_per_seq + j];
    if (block < 0 || block >= a.num_blocks) {
        if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(a.err, PKV_ERRBIT_BLOCK_ID);
        return;
    }
    const int low = max(first - j * bs, 0), high = min(len - j * bs, bs);  // the new rows
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int per_head = bs / ROWS;          // warps of a head
    const int h = blockIdx.y * (kWarps / per_head) + warp / per_head;
    const int row0 = (warp % per_head) * ROWS + lane / kTeam;
    const bool live = h < a.n_kv_heads;
    const int hc = live ? h : 0;
    const long long cell = block * a.n_kv_heads + hc;
    const long long token0 = static_cast<long long>(s) - first + j * bs;  // token of row 0
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const uint4 *src = static_cast<const uint4 *>(side ? a.v_new : a.k_new);
        const long long stride = (side ? a.v_stride : a.k_stride) / kPiece;
        uint4 x[kSteps];
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int row = row0 + i * kAt;
            x[i] = make_uint4(0, 0, 0, 0);
            if (live && row >= low && row < high)
                x[i] = __ldcs(src + (token0 + row) * stride + hc * kTeam + lane % kTeam);
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) top = fmaxf(top, top_of(x[i]));
#pragma unroll
        for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        float *scales = side ? a.v_scales : a.k_scales;
        const float had = live && low > 0 ? scales[cell] : 0.f;
        if (per_head > 1) {
            if (lane == 0) tops[side][warp] = top;
            __syncthreads();  // and every warp has read the old scale
            for (int w = 0; w < per_head; ++w) top = fmaxf(top, tops[side][warp / per_head * per_head + w]);
        } else {
            __syncwarp();
        }
        if (!live) continue;
        int power;
        const float scale = grown<KIND>(had, top, &power);
        uint2 *rows = static_cast<uint2 *>(side ? a.v_cache : a.k_cache) + cell * bs * kTeam + lane % kTeam;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int row = row0 + i * kAt;
            if (row >= low && row < high) rows[row * kTeam] = quantised<KIND>(x[i], scale);
        }
        if (power > 0)
            for (int row = row0; row < min(low, row0 + ROWS); row += kAt)
                rows[row * kTeam] = shrunk<KIND>(rows[row * kTeam], power);
        if (warp % per_head == 0 && lane == 0 && (low == 0 || scale != had)) scales[cell] = scale;
    }
}

template <int KIND, int D>
cudaError_t launch_append(const Q8AppendArgs &a, cudaStream_t stream) {
    if (a.max_q_len == 1) {
        const long long lanes = static_cast<long long>(a.num_seqs) * a.n_kv_heads * 2 * (D / kPiece);
        const long long blocks = (lanes + 127) / 128;
        if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
        return launch_pdl(q8_append_one_kernel<KIND, D>, dim3(static_cast<unsigned>(blocks)), dim3(128), 0,
                          stream, a);
    }
    const int rows = a.block_size == 256 ? 32 : 16;
    const int heads = kWarps / (a.block_size / rows);
    const long long slots = a.total / a.block_size + 2ll * a.num_seqs;
    const int groups = (a.n_kv_heads + heads - 1) / heads;
    if (slots > 0x7fffffffLL || groups > 65535) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(slots), static_cast<unsigned>(groups));
    if (rows == 32)
        return launch_pdl(q8_append_many_kernel<KIND, D, 32>, grid, dim3(kWarps * 32), 0, stream, a);
    return launch_pdl(q8_append_many_kernel<KIND, D, 16>, grid, dim3(kWarps * 32), 0, stream, a);
}

// --- read-back --------------------------------------------------------------

constexpr int kGatherThreads = 256, kGatherRows = 16;

// A CTA takes 16 output rows of every head: one thread a row finds its place in the
// cache, then each thread turns 16 codes into 32 bytes, rows next to each other in
// the block by neighbouring lanes.
template <int KIND, int D>
__global__ void __launch_bounds__(kGatherThreads) q8_gather_kernel(const Q8GatherArgs a) {
    constexpr int kLanes = D / 16;
    grid_dependency_wait();
    allow_dependent_launch();
    __shared__ int block_of[kGatherRows], row_of[kGatherRows];
    const long long first = static_cast<long long>(blockIdx.x) * kGatherRows;
    if (threadIdx.x < kGatherRows) {
        const long long r = first + threadIdx.x;
        int block = -1, row = 0;
        if (r < a.total && r >= a.start[0] && r < a.start[a.num_seqs]) {
            int lo = 0, hi = a.num_seqs;  // start[lo] <= r < start[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (a.start[mid] <= r) lo = mid; else hi = mid;
            }
            const long long t = r - a.start[lo];
            const long long j = t / a.block_size;
            if (t < 0 || j >= a.max_blocks_per_seq) {
                flag_error(a.err, PKV_ERRBIT_CONTEXT);
            } else {
                const int id = a.block_tables[static_cast<long long>(lo) * a.max_blocks_per_seq + j];
                if (id < 0 || id >= a.num_blocks) {
                    flag_error(a.err, PKV_ERRBIT_BLOCK_ID);
                } else {
                    block = id;
                    row = static_cast<int>(t - j * a.block_size);
                }
            }
        }
        block_of[threadIdx.x] = block;
        row_of[threadIdx.x] = row;
    }
    __syncthreads();
    const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes % kGatherRows;
    constexpr int kGroups = kGatherThreads / (kLanes * kGatherRows);  // (side, head) pairs at once
    const int block = block_of[row];
    if (block < 0) return;
    const long long r = first + row;
    for (int p = threadIdx.x / (kLanes * kGatherRows); p < 2 * a.n_kv_heads; p += kGroups) {
        const int side = p / a.n_kv_heads, h = p - side * a.n_kv_heads;
        const long long cell = static_cast<long long>(block) * a.n_kv_heads + h;
        const uint4 c = __ldcs(static_cast<const uint4 *>(side ? a.v_cache : a.k_cache) +
                               (cell * a.block_size + row_of[row]) * kLanes + lane);
        const float scale = (side ? a.v_scales : a.k_scales)[cell];
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t u = i % 2 ? q8_widen<KIND, 1>(w[i / 2]) : q8_widen<KIND, 0>(w[i / 2]);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
            // a NaN code stays NaN: the comparisons of the clamp are false for it
            float p0 = f.x * scale, p1 = f.y * scale;
            p0 = p0 > 65504.f ? 65504.f : p0 < -65504.f ? -65504.f : p0;
            p1 = p1 > 65504.f ? 65504.f : p1 < -65504.f ? -65504.f : p1;
            y[i] = pack_half2(p0, p1);
        }
        uint4 *dst = static_cast<uint4 *>(side ? a.v : a.k) + ((r * a.n_kv_heads + h) * kLanes + lane) * 2;
        __stcs(dst, make_uint4(y[0], y[1], y[2], y[3]));
        __stcs(dst + 1, make_uint4(y[4], y[5], y[6], y[7]));
    }
}

// --- block copy -------------------------------------------------------------

// A CTA a copy: the block's codes in 16-byte pieces, then its scales.
__global__ void __launch_bounds__(256) q8_copy_kernel(const Q8CopyArgs a) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int i = blockIdx.x;
    const int s = a.src[i], d = a.dst[i], n = a.tokens ? a.tokens[i] : a.block_size;
    if (s < 0 || s >= a.num_blocks || d < 0 || d >= a.num_blocks || n < 0 || n > a.block_size) {
        if (threadIdx.x == 0) flag_error(a.err, PKV_ERRBIT_SLOT);
        return;
    }
    const int lanes = a.head_dim / 16, per_head = a.block_size * lanes, whole = n * lanes;
    const long long from = static_cast<long long>(s) * a.n_kv_heads, to = static_cast<long long>(d) * a.n_kv_heads;
    uint4 *k = static_cast<uint4 *>(a.k_cache), *v = static_cast<uint4 *>(a.v_cache);
    for (int h = 0; h < a.n_kv_heads; ++h)
        for (int p = threadIdx.x; p < whole; p += 256) {
            k[(to + h) * per_head + p] = k[(from + h) * per_head + p];
            v[(to + h) * per_head + p] = v[(from + h) * per_head + p];
        }
    for (int h = threadIdx.x; h < a.n_kv_heads; h += 256) {
        a.k_scales[to + h] = a.k_scales[from + h];
        a.v_scales[to + h] = a.v_scales[from + h];
    }
}

}  // namespace

cudaError_t launch_q8_append(const Q8AppendArgs &a, int kind, cudaStream_t stream) {
    if (a.head_dim == 128)
        return kind == PKV_Q8_E4M3 ? launch_append<PKV_Q8_E4M3, 128>(a, stream)
                                   : launch_append<PKV_Q8_INT8, 128>(a, stream);
    return kind == PKV_Q8_E4M3 ? launch_append<PKV_Q8_E4M3, 64>(a, stream)
                               : launch_append<PKV_Q8_INT8, 64>(a, stream);
}

cudaError_t launch_q8_gather(const Q8GatherArgs &a, int kind, cudaStream_t stream) {
    const long long blocks = (a.total + kGatherRows - 1) / kGatherRows;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(blocks)), threads(kGatherThreads);
    if (a.head_dim == 128)
        return kind == PKV_Q8_E4M3
                   ? launch_pdl(q8_gather_kernel<PKV_Q8_E4M3, 128>, grid, threads, 0, stream, a)
                   : launch_pdl(q8_gather_kernel<PKV_Q8_INT8, 128>, grid, threads, 0, stream, a);
    return kind == PKV_Q8_E4M3
               ? launch_pdl(q8_gather_kernel<PKV_Q8_E4M3, 64>, grid, threads, 0, stream, a)
               : launch_pdl(q8_gather_kernel<PKV_Q8_INT8, 64>, grid, threads, 0, stream, a);
}

cudaError_t launch_q8_copy(const Q8CopyArgs &a, cudaStream_t stream) {
    return launch_pdl(q8_copy_kernel, dim3(static_cast<unsigned>(a.num_copies)), dim3(256), 0, stream, a);
}

}  // namespace pkv
