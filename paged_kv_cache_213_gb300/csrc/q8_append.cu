// q8_append.cu -- the append, the read-back and the block copy of the 8-bit
// caches with block scales (include/pagedkv_q8.h).
//
// Append.  The scale of a (block, head) needs the largest entry of all its new
// rows before the first code can be written, so whoever writes a block has all
// of them: a team of lanes holds the rows in registers, reduces their largest
// entry, and writes the codes from the same registers: one pass over memory.
// A token alone (decode) is a team of one row's lanes.
//
// Where a scale grows, the same lanes rewrite the rows that the block holds, one after another.  32
// tokens of 8 heads of 128, about half of a block's rows held (us): without growth 2.1 whatever the block;
// one scale of 16 growing, 16 rows a block, 3.5; every scale, 16 rows 3.9, 64 rows 8.6, 256 rows 27.
#include <cuda_fp16.h>

#include "f32x2.cuh"
#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "q8.h"
#include "q8_codes.cuh"

namespace pkv {
namespace {

// Entries of the head that one lane takes: 16 bytes of fp16, 8 of codes.
constexpr int kPiece = 8;

// The largest of 8 sizes |x|, as fp16 bits in either half of the result, and of another
// 8's; a NaN's bits where there is one.
__device__ __forceinline__ uint32_t top_bits(const uint4 &x, uint32_t other) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&x);
    __half2 top = *reinterpret_cast<const __half2 *>(&other);
#pragma unroll
    for (int i = 0; i < 4; ++i) top = __hmax2_nan(top, __habs2(h[i]));
    return *reinterpret_cast<const uint32_t *>(&top);
}

// The same over the finite values alone (sizes are ordered like their bits).
__device__ __forceinline__ uint32_t finite_top_bits(const uint4 &x, uint32_t other) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
        if (lo < 0x7c00u) other = __vmaxu2(other, lo);
        if (hi < 0x7c00u) other = __vmaxu2(other, hi);
    }
    return other;
}

// Largest finite |x| of N pieces, and whether some are not finite.
template <int N>
__device__ __forceinline__ float top_of(const uint4 (&x)[N], bool *special) {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) t = top_bits(x[i], t);
    *special = (t & 0xffffu) >= 0x7c00u || (t >> 16) >= 0x7c00u;
    if (*special) {
        t = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) t = finite_top_bits(x[i], t);
    }
    return __half2float(__ushort_as_half(static_cast<unsigned short>(max(t & 0xffffu, t >> 16))));
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

// What quantises by a scale: the divisor and its reciprocal (0: a scale that divide2 does
// not take).
struct Divisor {
    float s, inv;
    __device__ explicit Divisor(float scale) : s(scale > 0.f ? scale : 1.f) {
        inv = s >= 8.7e-19f && s <= 1.1e18f ? __frcp_rn(s) : 0.f;  // 2^-60, 2^60
    }
};

// Codes of 8 values.  PLAIN: they are finite, no larger than what the scale covers, and
// the divisor has a reciprocal.
template <int KIND, bool PLAIN>
__device__ __forceinline__ uint2 quantised(const uint4 &x, const Divisor &d) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&x);
    float2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        q[i] = PLAIN ? divide2_unsigned_zero(f, d.s, d.inv) : make_float2(__fdiv_rn(f.x, d.s), __fdiv_rn(f.y, d.s));
    }
    uint2 codes = make_uint2(q8_encode4<KIND, PLAIN>(q[0], q[1]), q8_encode4<KIND, PLAIN>(q[2], q[3]));
    if (PLAIN && KIND == PKV_Q8_E4M3) {  // the sign of a zero, with those that are there already
        codes.x |= __byte_perm(x.x, x.y, 0x7531) & 0x80808080u;
        codes.y |= __byte_perm(x.z, x.w, 0x7531) & 0x80808080u;
    }
    return codes;
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
        r[i] = q8_encode4<KIND>(make_float2(a.x * f, a.y * f), make_float2(b.x * f, b.y * f));
    }
    return make_uint2(r[0], r[1]);
}

// One token a sequence: a team of D / 8 lanes for each (sequence, head, K or V).  A launch
// and three loads in a row (length, block, scale): 32 x 8 heads of 128 2.1 us.
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
        const bool ok = n >= 0 && n <= 1 && n <= len && token >= 0 && token <= a.total - n &&
                        len <= static_cast<long long>(a.max_blocks_per_seq) * a.block_size;
        if (!ok && lane == 0 && h == 0 && side == 0) flag_error(a.err, PKV_ERRBIT_CONTEXT);
        live = ok && n == 1;
    }
    uint4 x[1] = {make_uint4(0, 0, 0, 0)};
    long long block = -1;
    int row = 0;
    if (live) {
        const uint4 *src = static_cast<const uint4 *>(side ? a.v_new : a.k_new);
        x[0] = __ldcs(src + (token * (side ? a.v_stride : a.k_stride) + h * D) / kPiece + lane);
        const int j = (len - 1) / a.block_size;
        row = (len - 1) - j * a.block_size;
        block = a.block_tables[static_cast<long long>(b) * a.max_blocks_per_seq + j];
        if (block < 0 || block >= a.num_blocks) {
            if (lane == 0 && h == 0 && side == 0) flag_error(a.err, PKV_ERRBIT_BLOCK_ID);
            live = false;
        }
    }
    const long long cell = block * a.n_kv_heads + h;
    float *scales = side ? a.v_scales : a.k_scales;
    const float had = live && row > 0 ? scales[cell] : 0.f;
    bool special;
    float top = top_of(x, &special);
#pragma unroll
    for (int d = kTeam / 2; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    __syncwarp();  // every lane has read the old scale, which one lane writes below
    if (!live) return;
    int power;
    const float scale = grown<KIND>(had, top, &power);
    uint2 *rows = static_cast<uint2 *>(side ? a.v_cache : a.k_cache) + cell * a.block_size * kTeam + lane;
    const Divisor divisor(scale);
    rows[row * kTeam] = special || divisor.inv == 0.f ? quantised<KIND, false>(x[0], divisor)
                                                      : quantised<KIND, true>(x[0], divisor);
    if (power > 0)
        for (int r = 0; r < row; ++r) rows[r * kTeam] = shrunk<KIND>(rows[r * kTeam], power);
    if (lane == 0 && (row == 0 || scale != had)) scales[cell] = scale;
}

// Several tokens a sequence.  A CTA takes K or V of one block that a sequence touches, for
// kWarps * 16 / block_size heads (one head from kWarps * 16 rows on), its warps 16 rows
// each (32 or 64 at 128 or 256 rows a block); the warps of a head exchange their largest entries.
//
// Which block: the blocks of sequence b get the numbers from start[b] / bs + 2 b on.
// A run of n tokens touches at most n / bs + 2 blocks (rounded down), so the ranges do
// not meet, and a CTA finds its sequence without a sum over the ones before.  Where starts
// decrease (flagged) they may: the CTA then takes those that are in bounds one by one.
//
// 8 CTAs an SM, each with its rows on the way before it knows the scale.  5 prompts of 411
// to 2903 tokens, 8 heads of 128 (51 MB): 12.8 us, 4.0 TB/s; by instructions (half of the issue
// slots) and by starts and ends, which a transfer of 7.5 us does not hide.  2 or 8 warps a CTA,
// 40 warps an SM: 12.9, 13.4, 12.9; 24 warps an SM 15.2.
// (At 32 and 64 rows a warp: the CTAs that its registers leave room for without spills.)
constexpr int kWarps = 4;

template <int KIND, int D, int ROWS>  // rows of a warp
__global__ void __launch_bounds__(kWarps * 32, ROWS == 16 ? 8 : ROWS * D == 32 * 64 ? 5 : ROWS * D == 64 * 128 ? 2 : 4)
    q8_append_many_kernel(const Q8AppendArgs a) {
    constexpr int kTeam = D / kPiece;        // lanes of a row
    constexpr int kAt = 32 / kTeam;          // rows of one load
    constexpr int kSteps = ROWS / kAt;
    grid_dependency_wait();
    allow_dependent_launch();
    struct Found {
        int b, start, n, len;
        int more;  // its finder found others too
    };
    __shared__ Found found;
    __shared__ int owner;
    __shared__ float tops[kWarps];
    const int v = blockIdx.x;  // at most total / 16 + 2 * 2048
    const int bs = a.block_size, bs_log2 = __ffs(bs) - 1, side = blockIdx.z;
    const bool reports = blockIdx.y == 0 && side == 0 && threadIdx.x == 0;

    auto append = [&](const Found f) {
        const int slot = v - ((f.start >> bs_log2) + 2 * f.b);
        if (f.n > a.max_q_len || f.n > f.len || f.len > static_cast<long long>(a.max_blocks_per_seq) * bs) {
            if (reports && slot == 0) flag_error(a.err, PKV_ERRBIT_CONTEXT);
            return;
        }
        const int first = f.len - f.n, j = (first >> bs_log2) + slot;
        if (static_cast<long long>(j) * bs >= f.len) return;
        const long long block = a.block_tables[static_cast<long long>(f.b) * a.max_blocks_per_seq + j];
        const int low = max(first - j * bs, 0), high = min(f.len - j * bs, bs);  // the new rows
        int tid;  // read anew: rows and addresses are not kept for a second sequence
        asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
        const int warp = tid / 32, lane = tid % 32;
        const int per_head = bs / ROWS;          // warps of a head
        const int h = blockIdx.y * (kWarps / per_head) + warp / per_head;
        const int row0 = (warp % per_head) * ROWS + lane / kTeam;
        const bool live = h < a.n_kv_heads;
        const int hc = live ? h : 0;
        // the tokens are read while the block's number is on its way
        const uint4 *src = static_cast<const uint4 *>(side ? a.v_new : a.k_new) + hc * kTeam + lane % kTeam;
        const long long stride = (side ? a.v_stride : a.k_stride) / kPiece;
        const long long token0 = static_cast<long long>(f.start) - first + j * bs;  // token of row 0
        uint4 x[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int row = row0 + i * kAt;
            x[i] = make_uint4(0, 0, 0, 0);
            if (live && row >= low && row < high) x[i] = __ldcs(src + (token0 + row) * stride);
        }
        if (block < 0 || block >= a.num_blocks) {
            if (reports) flag_error(a.err, PKV_ERRBIT_BLOCK_ID);
            return;
        }
        const long long cell = block * a.n_kv_heads + hc;
        float *scales = side ? a.v_scales : a.k_scales;
        const float had = live && low > 0 ? scales[cell] : 0.f;
        bool special;
        float top = top_of(x, &special);
#pragma unroll
        for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        if (per_head > 1) {
            if (lane == 0) tops[warp] = top;
            __syncthreads();  // and every warp has read the old scale
            for (int w = 0; w < per_head; ++w) top = fmaxf(top, tops[warp / per_head * per_head + w]);
        }
        if (!live) return;
        __syncwarp();
        int power;
        const float scale = grown<KIND>(had, top, &power);
        const Divisor divisor(scale);
        uint2 *rows = static_cast<uint2 *>(side ? a.v_cache : a.k_cache) + cell * bs * kTeam + lane % kTeam;
        if (!special && divisor.inv != 0.f) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int row = row0 + i * kAt;
                if (row >= low && row < high) rows[row * kTeam] = quantised<KIND, true>(x[i], divisor);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int row = row0 + i * kAt;
                if (row >= low && row < high) rows[row * kTeam] = quantised<KIND, false>(x[i], divisor);
            }
        }
        if (power > 0)
            for (int row = row0; row < min(low, row0 - lane / kTeam + ROWS); row += kAt)
                rows[row * kTeam] = shrunk<KIND>(rows[row * kTeam], power);
        if (warp % per_head == 0 && lane == 0 && (low == 0 || scale != had)) scales[cell] = scale;
    };

    for (int last = -1;;) {  // the sequences behind it that have this number: one, with starts in order
        Found mine{-1, 0, 0, 0, 0};
        for (int b = threadIdx.x; b < a.num_seqs; b += kWarps * 32) {
            const int s = a.query_start[b], e = a.query_start[b + 1], len = a.context_lens[b];
            if (s < 0 || e < s || e > a.total ||
                (e == s && (len < 0 || len > static_cast<long long>(a.max_blocks_per_seq) * bs))) {
                if (v == 0 && blockIdx.y == 0 && side == 0) flag_error(a.err, PKV_ERRBIT_CONTEXT);
                continue;
            }
            const int low = (s >> bs_log2) + 2 * b, end = (e >> bs_log2) + 2 * (b + 1);
            if (v < low || v >= end || b <= last || e == s) continue;
            if (mine.b < 0)
                mine = Found{b, s, e - s, len, 0};
            else
                mine.more = 1;
        }
        if (mine.b >= 0) found = mine;
        const int finders = __syncthreads_count(mine.b >= 0);
        if (finders == 0) return;
        if (finders > 1) {  // what they wrote may be mixed: the first sequence's finder writes again
            if (threadIdx.x == 0) owner = a.num_seqs;
            __syncthreads();
            if (mine.b >= 0) atomicMin(&owner, mine.b);
            __syncthreads();
            if (mine.b == owner) found = mine;
            __syncthreads();
        }
        const Found f = found;
        append(f);
        if (finders == 1 && !f.more) return;
        last = f.b;
        __syncthreads();
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
    const int rows = a.block_size <= kWarps * 16 ? 16 : a.block_size / kWarps;
    const int heads = kWarps * rows / a.block_size;
    const long long slots = a.total / a.block_size + 2ll * a.num_seqs;
    const int groups = (a.n_kv_heads + heads - 1) / heads;
    if (slots > 0x7fffffffLL || groups > 65535) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(slots), static_cast<unsigned>(groups), 2), threads(kWarps * 32);
    if (rows == 64) return launch_pdl(q8_append_many_kernel<KIND, D, 64>, grid, threads, 0, stream, a);
    if (rows == 32) return launch_pdl(q8_append_many_kernel<KIND, D, 32>, grid, threads, 0, stream, a);
    return launch_pdl(q8_append_many_kernel<KIND, D, 16>, grid, threads, 0, stream, a);
}

// --- read-back --------------------------------------------------------------

constexpr int kGatherThreads = 256;

// A CTA takes ROWS output rows of every head.  Each thread asks whether its sequences own
// some of them (no search, whose steps would wait for one another), one thread a row
// looks the row's block up, then each thread turns 16 codes into 32 bytes, rows next
// to each other in the block by neighbouring lanes.
// 8 sequences of 2000 to 16000 tokens, 8 heads of 128 (442 MB): 70.1 us, 6.3 TB/s: memory.
// (The bound of one CTA lets the compiler take 48 registers and keep both loads in flight; at the
// 32 that it takes without, 72000 rows take 82.6 us.)
template <int KIND, int D, int ROWS>
__global__ void __launch_bounds__(kGatherThreads, 1) q8_gather_kernel(const Q8GatherArgs a) {
    constexpr int kLanes = D / 16;
    grid_dependency_wait();
    allow_dependent_launch();
    __shared__ int seq_of[ROWS], block_of[ROWS], row_of[ROWS];
    const long long first = static_cast<long long>(blockIdx.x) * ROWS;
    if (threadIdx.x < ROWS) seq_of[threadIdx.x] = -1;
    __syncthreads();
    for (int b = threadIdx.x; b < a.num_seqs; b += kGatherThreads) {
        const long long s = a.start[b], e = a.start[b + 1];
        if (s < 0) continue;
        for (long long r = max(s, first); r < min(e, first + ROWS); ++r) {
            seq_of[r - first] = b;
            row_of[r - first] = static_cast<int>(r - s);
        }
    }
    __syncthreads();
    if (threadIdx.x < ROWS) {
        const int b = seq_of[threadIdx.x];
        int block = -1, row = 0;
        if (b >= 0 && first + threadIdx.x < a.total) {
            const int t = row_of[threadIdx.x], j = t / a.block_size;
            if (j >= a.max_blocks_per_seq) {
                flag_error(a.err, PKV_ERRBIT_CONTEXT);
            } else {
                block = a.block_tables[static_cast<long long>(b) * a.max_blocks_per_seq + j];
                row = t - j * a.block_size;
                if (block < 0 || block >= a.num_blocks) {
                    flag_error(a.err, PKV_ERRBIT_BLOCK_ID);
                    block = -1;
                }
            }
        }
        block_of[threadIdx.x] = block;
        row_of[threadIdx.x] = row;
    }
    __syncthreads();
    const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes % ROWS;
    constexpr int kGroups = kGatherThreads / (kLanes * ROWS);  // (side, head) pairs at once
    constexpr int kAtOnce = 2;  // and in flight a thread (1: 73.4 us, 4: 87, with 8 x 2000-16000 tokens; this 70.1)
    const int block = block_of[row];
    if (block < 0) return;
    const long long r = first + row;
    for (int p0 = threadIdx.x / (kLanes * ROWS); p0 < 2 * a.n_kv_heads; p0 += kGroups * kAtOnce) {
        uint4 c[kAtOnce];
        float scale[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int p = p0 + i * kGroups, side = p >= a.n_kv_heads, h = side ? p - a.n_kv_heads : p;
            if (p >= 2 * a.n_kv_heads) continue;
            const long long cell = static_cast<long long>(block) * a.n_kv_heads + h;
            c[i] = __ldcs(static_cast<const uint4 *>(side ? a.v_cache : a.k_cache) +
                          (cell * a.block_size + row_of[row]) * kLanes + lane);
            scale[i] = (side ? a.v_scales : a.k_scales)[cell];
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int p = p0 + i * kGroups, side = p >= a.n_kv_heads, h = side ? p - a.n_kv_heads : p;
            if (p >= 2 * a.n_kv_heads) continue;
            const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t u = k % 2 ? q8_widen<KIND, 1>(w[k / 2]) : q8_widen<KIND, 0>(w[k / 2]);
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
                // rounded to fp32 here and to fp16 below (a product has 28 or 31 bits: one rounding alone
                // would take its residual as well, for one entry in 20000).  A NaN code stays NaN: the
                // comparisons of the clamp are false for it
                float p0 = f.x * scale[i], p1 = f.y * scale[i];
                p0 = p0 > 65504.f ? 65504.f : p0 < -65504.f ? -65504.f : p0;
                p1 = p1 > 65504.f ? 65504.f : p1 < -65504.f ? -65504.f : p1;
                y[k] = pack_half2(p0, p1);
            }
            uint4 *dst = static_cast<uint4 *>(side ? a.v : a.k) + ((r * a.n_kv_heads + h) * kLanes + lane) * 2;
            __stcs(dst, make_uint4(y[0], y[1], y[2], y[3]));
            __stcs(dst + 1, make_uint4(y[4], y[5], y[6], y[7]));
        }
    }
}

// --- block copy -------------------------------------------------------------

// A CTA a copy: the block's codes in 16-byte pieces, then its scales.  For the few copies of a
// step's forks, where the launch is all there is.
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

namespace {

template <int KIND, int D>
cudaError_t launch_gather(const Q8GatherArgs &a, cudaStream_t stream) {
    // 16 rows a CTA, or 8 where those are less than two CTAs for each of 152 SMs (1160 rows of 8
    // heads: 3.5 us, with 16 rows 5.1; 72000 rows: 73.8 us with 8 rows, 70.1 with 16)
    const bool few = a.total <= 16 * 2 * 152;
    const long long blocks = (a.total + (few ? 7 : 15)) / (few ? 8 : 16);
    const dim3 grid(static_cast<unsigned>(blocks)), threads(kGatherThreads);
    return few ? launch_pdl(q8_gather_kernel<KIND, D, 8>, grid, threads, 0, stream, a)
               : launch_pdl(q8_gather_kernel<KIND, D, 16>, grid, threads, 0, stream, a);
}

}  // namespace

cudaError_t launch_q8_gather(const Q8GatherArgs &a, int kind, cudaStream_t stream) {
    if (a.head_dim == 128)
        return kind == PKV_Q8_E4M3 ? launch_gather<PKV_Q8_E4M3, 128>(a, stream)
                                   : launch_gather<PKV_Q8_INT8, 128>(a, stream);
    return kind == PKV_Q8_E4M3 ? launch_gather<PKV_Q8_E4M3, 64>(a, stream)
                               : launch_gather<PKV_Q8_INT8, 64>(a, stream);
}

cudaError_t launch_q8_copy(const Q8CopyArgs &a, cudaStream_t stream) {
    return launch_pdl(q8_copy_kernel, dim3(static_cast<unsigned>(a.num_copies)), dim3(256), 0, stream, a);
}

}  // namespace pkv
