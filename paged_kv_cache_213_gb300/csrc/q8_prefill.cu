// q8_prefill.cu -- attention over the 8-bit caches with block scales for many query rows
// of a KV head: chunks of prompts, drafts to verify (paged_decode_attention_q8).
//
// An item is two tiles of 128 query rows (tokens x heads of a group) of one KV head.  For a
// step of 64 keys, codes K, V widened to fp16 (exact) in shared memory:
//   S [128 x 64] = Q K^T
//   y = 2^(S f - r)          f: the key's block scale * scale * log2 e; r: the row's reference
//   O += (y v / w) V         v: the key's block scale; w: the item's V reference
// with S, O and P = y v / w in TMEM: P (fp16) takes the place of its own S and is the first
// operand of the second product.  r moves only when a logit is 2^kLag above it, w when the
// largest v of a step leaves [w / 64, 16 w]; O is then rescaled in TMEM by the thread that
// owns the row.  The result is O w / l, l the sum of y before its rounding.
//
// Roles: two warpgroups of softmax, a tile each, a row a thread; one of converters, which
// load codes into registers two steps ahead, widen them and store them in the products'
// layout; a warp of products for each tile.  A tile has two places for S, so the scores of
// the next step are there when the softmax of one is done.  (With one place, and steps of
// 128 keys, softmax and products of a tile took turns: 113 us for the chunks below.)
//
// Split.  The (sequence, head, pair of tiles, step) units are cut into equal ranges, one
// per SM; items that several CTAs hold leave records, and the last to arrive joins them.
//
// Measured: 3 chunks of 150 to 700 tokens behind 1800 to 2500, 32 query heads on 8 of 128 (47
// GFLOP): 63.1 us, 0.75 PFLOP/s.  A step takes about 2200 cycles, in which the tensor pipe is busy
// 980: the softmax of a row's 64 keys is the chain.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <atomic>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "q8.h"
#include "q8_codes.cuh"
#include "rope_latent.h"
#include "tc05.cuh"

namespace pkv {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

namespace {

constexpr int kRows = 128, kKeys = 64;  // of a tile, of a step
static_assert(kQ8MaxGroup <= kRows, "a token's rows are in one tile");
constexpr int kPair = 2 * kRows;
constexpr int kGroups = kKeys / 16;      // pieces of 16 keys, each of one block
constexpr int kThreads = 512;  // 8 warps of softmax, 4 of converters, 2 of products, 1 of queries, an idle one
constexpr int kQPlane = kRows * 128, kPlane = kKeys * 128;  // rows of 64 fp16, swizzled
constexpr float kLag = 8.f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kStages = 4;  // of the ring of K and V
// Most waits last a step, two a piece: a tile's queries wait for the scores of the piece before, and
// the softmax of a tile without rows for the next piece's.  2^25 tokens are 0.6 s at 1.1 us a
// step, within what a wait may take.
constexpr int kMaxTokens = 1 << 25;

template <int D>
struct Cfg {
    static constexpr int kPlanes = D / 64;
    static constexpr int kQ = kPlanes * kQPlane;      // bytes of a tile's queries
    static constexpr int kHalf = kPlanes * kPlane;    // of a step's K or V
    static constexpr int kBytes = 2 * kQ + 2 * kStages * kHalf;  // queries, K ring, V ring
    static constexpr size_t smem(int seqs) { return kBytes + (static_cast<size_t>(seqs) * 3 + 2) * 4; }
};

// A piece that other CTAs share, to be joined if this warp was the last to arrive with its rows.
struct Share {
    int b, h, p;
    int from, parts, before;  // CTAs from, parts of them; how many had arrived
};

// What a softmax warp knows of its piece, here while it goes through the steps: that loop has
// 64 logits in registers and is slower with each other one that it has to leave room for (69.3
// us for the chunks above, 63.4 with this).
struct Piece {
    int u, first, n, f, mine, shares, b, h, p, steps;
};

struct Roles {
    Share todo[8][2];
    Piece keep[8];
    uint64_t q_full[2], q_empty[2], o_free[2], drained[2];
    // Of a tile's even and odd steps.  With the scores two steps ahead, a warp of softmax may be
    // a step ahead of the others, whose arrivals it must not make up for, and done with a
    // step when the outputs of the one before are not: a wait that names its phase by
    // parity alone would take them for the step's own.
    uint64_t s_full[2][2], p_ready[2][2], pv_done[2][2];
    uint64_t full[kStages], empty[kStages];
    // Of a step's keys: the logits' factor and the V scale; a stage is written again when the
    // outputs of its step are done, and so its softmax.
    float f[kStages][kGroups], v[kStages][kGroups];
    uint32_t tmem;
    int queries[2];  // tiles of queries copied
    int stop;
    int sums[kThreads / 32];
};

struct Batch {
    const int *cum, *len, *start;  // units before a sequence, its tokens, its first query row
};

// A place in the order of the units: sequence, KV head, pair of row tiles, step.
struct Place {
    int b, h, p, j;
    int steps;  // of the pair

    // Keys that the tokens of the sequence up to number `tok` attend.
    static __device__ int keys(const Batch &t, int b, int tok) {
        const int n = t.start[b + 1] - t.start[b];
        return t.len[b] - n + 1 + min(tok, n - 1);
    }
    static __device__ int steps_of(const Batch &t, const Q8AttentionArgs &a, int b, int p) {
        return (keys(t, b, 2 * (p + 1) * a.tile_tokens - 1) + kKeys - 1) / kKeys;
    }
    static __device__ int pairs(const Batch &t, const Q8AttentionArgs &a, int b) {
        return (t.start[b + 1] - t.start[b] + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
    }
    __device__ void find(const Batch &t, const Q8AttentionArgs &a, int u) {
        int lo = 0, hi = a.num_seqs;  // cum[lo] <= u < cum[hi]
#pragma unroll 1
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (t.cum[mid] <= u) lo = mid; else hi = mid;
        }
        b = lo;
        const int of_head = (t.cum[b + 1] - t.cum[b]) / a.n_kv_heads;
        j = u - t.cum[b];
        h = j / of_head;
        j -= h * of_head;
        p = 0;
#pragma unroll 1
        while (j >= (steps = steps_of(t, a, b, p))) j -= steps, ++p;
    }
    // The first unit of the next pair.
    __device__ void next(const Batch &t, const Q8AttentionArgs &a) {
        j = 0;
        if (++p == pairs(t, a, b)) {
            p = 0;
            if (++h == a.n_kv_heads) {
                h = 0;
#pragma unroll 1
                do ++b; while (b < a.num_seqs && t.cum[b + 1] == t.cum[b]);
                if (b >= a.num_seqs) return;
            }
        }
        steps = steps_of(t, a, b, p);
    }
    // The steps of tile t of the pair; 0: it has no rows.
    __device__ int steps_of_tile(const Batch &t, const Q8AttentionArgs &a, int tile) const {
        const int tok = (2 * p + tile) * a.tile_tokens;
        if (tok >= t.start[b + 1] - t.start[b]) return 0;
        return (keys(t, b, tok + a.tile_tokens - 1) + kKeys - 1) / kKeys;
    }
};

// CTA c of n has the units [cut(c), cut(c + 1)).
struct Ranges {
    int size, larger;
    __device__ Ranges(int total, int n) : size(total / n), larger(total - size * n) {}
    __device__ int start(int i) const { return size * i + min(i, larger); }
    __device__ int of(int x) const {
        const int split = larger * (size + 1);
        return x < split ? x / (size + 1) : larger + (x - split) / max(size, 1);
    }
};

__device__ __forceinline__ int divided(int x, const Q8Divide &d) {
    return static_cast<int>(static_cast<unsigned long long>(static_cast<unsigned>(x)) * d.mul >> d.shift);
}

// A thread's row among the pair's: its token, and its head in the group.  Rows behind the
// tile's tokens (where the group does not divide 128) are no token's.
struct Row {
    int in_pair, tok, head;
    __device__ Row(const Q8AttentionArgs &a, int row) : in_pair(row) {
        const int group = a.n_q_heads / a.n_kv_heads, t = row / kRows, i = row % kRows;
        const int tok_in = divided(i, a.by_group);
        head = i - tok_in * group;
        tok = tok_in < a.tile_tokens ? t * a.tile_tokens + tok_in : 1 << 29;
    }
    __device__ long long out_row(const Batch &t, const Q8AttentionArgs &a, int b, int h, int p) const {
        return static_cast<long long>(t.start[b] + 2 * p * a.tile_tokens + tok) * a.n_q_heads +
               h * (a.n_q_heads / a.n_kv_heads) + head;
    }
};

// A piece of 16 bytes in the products' layout: row `row` of a plane, piece q of 8.
__device__ __forceinline__ int swizzled(int row, int q) { return row * 128 + ((q ^ (row & 7)) << 4); }

template <int KIND, int D>
__global__ void __launch_bounds__(kThreads, 1) q8_prefill_kernel(const Q8AttentionArgs a,
                                                                const __grid_constant__ CUtensorMap q_map) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char base[];
    __shared__ __align__(16) Roles sh;
    int *cum = reinterpret_cast<int *>(base + C::kBytes), *len = cum + a.num_seqs + 1, *start = len + a.num_seqs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = a.n_q_heads / a.n_kv_heads;

    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sh.q_full[t], 1);
            mbar_init(&sh.q_empty[t], 1);
            mbar_init(&sh.s_full[t][0], 2);
            mbar_init(&sh.s_full[t][1], 2);
            mbar_init(&sh.o_free[t], 4);
            mbar_init(&sh.p_ready[t][0], 4);
            mbar_init(&sh.p_ready[t][1], 4);
            mbar_init(&sh.pv_done[t][0], 1);
            mbar_init(&sh.pv_done[t][1], 1);
            mbar_init(&sh.drained[t], 1);
        }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 4);
            mbar_init(&sh.empty[s], 2);
        }
        sh.stop = sh.queries[0] = sh.queries[1] = 0;
        fence_barrier_init();
    }
    if (warp == 12) tmem_alloc(&sh.tmem, 512);
    if (threadIdx.x == 0) prefetch_tmap(&q_map);
    tc_fence_before();
    grid_dependency_wait();
    allow_dependent_launch();

    // --- the batch's units
    const Batch t{cum, len, start};
    int total = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.num_seqs; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int n = 0;
        if (b < a.num_seqs) {
            int l = a.context_lens[b], s = b;
            n = 1;
            if (a.query_start) {
                s = a.query_start[b];
                n = a.query_start[b + 1] - s;
            } else if (l == 0) {
                n = 0;
            }
            const bool ok = n >= 0 && n <= a.max_q_len && n <= l && s >= 0 && s <= a.total_q - n &&
                            l <= a.max_context_len;
            if (!ok && blockIdx.x == 0) flag_error(a.err, PKV_ERRBIT_CONTEXT);
            len[b] = l;
            start[b] = s;
            if (b == a.num_seqs - 1) start[b + 1] = s + n;
            if (!ok) n = 0;
        }
        __syncthreads();
        int units = 0;
        if (n > 0) {
#pragma unroll 1
            for (int tok = 0; tok < n; tok += 2 * a.tile_tokens)
                units += (len[b] - n + kKeys + min(tok + 2 * a.tile_tokens, n) - 1) / kKeys;
            units *= a.n_kv_heads;
        }
        int upto = units;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int z = __shfl_up_sync(~0u, upto, d);
            if (lane >= d) upto += z;
        }
        if (lane == 31) sh.sums[warp] = upto;
        __syncthreads();
        int before = total;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const int x = sh.sums[w];
            if (w < warp) before += x;
            total += x;
        }
        if (b < a.num_seqs) cum[b] = before + upto - units;
        __syncthreads();
    }
    if (threadIdx.x == 0) cum[a.num_seqs] = total;
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    volatile int *stop = &sh.stop;
    // TMEM columns: S of tile t at 128 t and 128 t + 64 (P in its first half), O at 256 + 128 t

    const int ctas = min(static_cast<int>(gridDim.x), max(1, total));
    const Ranges ranges(total, ctas);
    const int cta = blockIdx.x;
    const int U0 = cta < ctas ? ranges.start(cta) : 0, U1 = cta < ctas ? ranges.start(cta + 1) : 0;
    if (!a.query_start) {  // one token a sequence: an empty one has a result
#pragma unroll 1
        for (int b = cta; b < a.num_seqs; b += gridDim.x) {
            if (len[b] != 0) continue;
            uint4 *o = static_cast<uint4 *>(a.out) + static_cast<long long>(b) * a.n_q_heads * (D / 8);
#pragma unroll 1
            for (int i = threadIdx.x; i < a.n_q_heads * (D / 8); i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
            if (a.lse_out)
#pragma unroll 1
                for (int i = threadIdx.x; i < a.n_q_heads; i += kThreads)
                    a.lse_out[static_cast<long long>(b) * a.n_q_heads + i] = -INFINITY;
        }
    }
    Place at{};
    if (U0 < U1) at.find(t, a, U0);

    if (warp == 14) {
        // --- queries: a box of a tile's tokens and heads for each 64 columns.  Their place is
        // free when the scores of the tile's piece before are done
        if (elect_one()) {
            const int tokens = a.tile_tokens, bytes = C::kPlanes * tokens * group * 128;
            int pc[2] = {0, 0};
            bool ok = true;
#pragma unroll 1
            for (int u = U0; ok && u < U1; at.next(t, a)) {
                const int n = min(at.steps - at.j, U1 - u);
                u += n;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (!ok || min(at.steps_of_tile(t, a, w) - at.j, n) <= 0) continue;
                    ok = wait_or_stop(&sh.q_empty[w], (pc[w] & 1) ^ 1, stop);
                    if (!ok) break;
                    ++pc[w];
                    mbar_arrive_expect_tx(&sh.q_full[w], bytes);
#pragma unroll
                    for (int p = 0; p < C::kPlanes; ++p)
                        tma_load_3d(base + w * C::kQ + p * kQPlane, &q_map, 64 * p, at.h * group,
                                    start[at.b] + (2 * at.p + w) * tokens, &sh.q_full[w]);
                }
            }
            sh.queries[0] = pc[0];
            sh.queries[1] = pc[1];
        }
    } else if (warp >= 12) {
        // --- products ---
        if (warp < 14 && elect_one()) {
            const int w = warp - 12;  // the tile
            constexpr uint32_t ds = mma_desc(kRows, kKeys, false, false), dpv = mma_desc(kRows, D, false, true);
            const uint32_t kv = smem_addr(base) + 2 * C::kQ, ts = tmem + 128 * w;
            const uint64_t qd = smem_desc(smem_addr(base) + w * C::kQ, 1024, 0);
            int f = 0, ss = 0, sc = 0, pc = 0;  // steps so far; this tile's scores, weights and pieces
            bool ok = U0 == U1 || first_wait(&sh.full[0], 0, a.first_wait_polls, stop);
#pragma unroll 1
            for (int u = U0; ok && u < U1; at.next(t, a)) {
                const int n = min(at.steps - at.j, U1 - u);  // steps of this piece, and of its tile
                const int mine = max(0, min(at.steps_of_tile(t, a, w) - at.j, n));
                u += n;
#pragma unroll 1
                for (int i = 0; i < n + 2; ++i) {  // outputs of step i - 2, scores of step i in their S's place
                    if (i >= 2) {
                        const int j = i - 2, vf = f + j;
                        if (j < mine) {
                            if (j == 0 && pc > 0) ok = wait_or_stop(&sh.o_free[w], (pc - 1) & 1, stop);
                            ok = ok && wait_or_stop(&sh.p_ready[w][sc & 1], (sc >> 1) & 1, stop);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t vd = smem_desc(kv + (2 * (vf % kStages) + 1) * C::kHalf, 1024, kPlane);
#pragma unroll
                            for (int k = 0; k < kKeys / 16; ++k)
                                mma_ts(ts + 256, ts + 64 * (sc & 1) + 8 * k, vd + k * 128, dpv, j > 0 || k > 0);
                            mma_commit(&sh.pv_done[w][sc & 1]);
                            ++sc;
                        }
                        mma_commit(&sh.empty[vf % kStages]);
                    }
                    if (i < n) {
                        const int kf = f + i;
                        ok = wait_or_stop(&sh.full[kf % kStages], (kf / kStages) & 1, stop);
                        if (ok && i < mine) {
                            if (i == 0) ok = wait_or_stop(&sh.q_full[w], pc & 1, stop);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t kd = smem_desc(kv + 2 * (kf % kStages) * C::kHalf, 1024, 0);
#pragma unroll
                            for (int k = 0; k < 4 * C::kPlanes; ++k)
                                mma_ss(ts + 64 * (ss & 1), qd + (k / 4) * (kQPlane / 16) + (k % 4) * 2,
                                       kd + (k / 4) * (kPlane / 16) + (k % 4) * 2, ds, k > 0);
                            mma_commit(&sh.s_full[w][ss & 1]);
                            // what this thread has seen (the scales) is seen there too
                            mbar_arrive(&sh.s_full[w][ss & 1]);
                            ++ss;
                            if (i + 1 == mine) mma_commit(&sh.q_empty[w]);
                        }
                        if (!ok) break;
                    }
                }
                f += n;
                if (mine > 0) ++pc;
            }
            // nothing of the tensor core is left in flight when TMEM is freed
            mma_commit(&sh.drained[w]);
            mbar_wait_bounded(&sh.drained[w], 0);
        }
    } else if (warp >= 8) {
        // --- converters ---
        const int w = warp - 8;  // its 16 keys of a step
        constexpr int kAt = 32 / (4 * C::kPlanes), kLoads = 16 / kAt;  // rows of a load, loads of 16 rows
        // A lane's 16 codes of a row become pieces 2 x and 2 x + 1 of a plane.  Eight lanes have
        // two rows of one plane, whose swizzles differ in the lowest bit: no bank twice.
        const int plane = lane / 16 * (C::kPlanes - 1), x4 = lane % 4;
        const int row0 = C::kPlanes == 2 ? lane / 4 % 4 : lane / 4;
        const int bs16_log2 = __ffs(a.block_size / 16) - 1;
        const int code_at = row0 * D + plane * 64 + x4 * 16;
        const unsigned char *kc = static_cast<const unsigned char *>(a.k_cache) + code_at;
        const unsigned char *vc = static_cast<const unsigned char *>(a.v_cache) + code_at;
        // where the lane stores, for loads of even and odd number (the others lie 8 rows on)
        int to[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                to[i][e] = plane * kPlane + swizzled(w * 16 + (i * kAt & 7) + row0, 2 * x4 + e);
        const float scale = fmaxf(fabsf(a.scale_log2), 1e-30f);
        unsigned char *ring = base + 2 * C::kQ;
        int f = 0;  // steps so far
        bool ok = true;
#pragma unroll 1
        for (int u = U0; ok && u < U1; at.next(t, a)) {
            const int n = min(at.steps - at.j, U1 - u);
            u += n;
            const int L = len[at.b];
            const int *table = a.block_tables + static_cast<long long>(at.b) * a.max_blocks_per_seq;
            // lane i knows the cache piece (16 rows) of step from + i for this warp's keys; two
            // batches of 32 steps
            auto pieces = [&](int from) {
                const int g = (at.j + from + lane) * kGroups + w;  // of the sequence
                unsigned piece = 0;
                if (from + lane < n && g * 16 < L) {
                    const int id = table[g >> bs16_log2];
                    if (id < 0 || id >= a.num_blocks)
                        flag_error(a.err, PKV_ERRBIT_BLOCK_ID);
                    else
                        piece = (static_cast<unsigned>(id) * a.n_kv_heads + at.h << bs16_log2) +
                                (g & ((1 << bs16_log2) - 1));
                }
                return piece;
            };
            unsigned now = pieces(0), next = pieces(32);
            uint4 xk[2][kLoads], xv[2][kLoads];  // codes of the next two steps, on their way
            float ks[2], vs[2];
            auto load = [&](int e, int j) {  // step j, all in one go
                if (j >= n) return;
                if (j > 0 && (j & 31) == 0) {
                    now = next;
                    next = pieces(j + 32);
                }
                const unsigned piece = __shfl_sync(~0u, now, j & 31);
                const long long src = static_cast<long long>(piece) * (16 * D);
#pragma unroll
                for (int i = 0; i < kLoads; ++i) xk[e][i] = __ldcg(reinterpret_cast<const uint4 *>(kc + src + i * kAt * D));
#pragma unroll
                for (int i = 0; i < kLoads; ++i) xv[e][i] = __ldcg(reinterpret_cast<const uint4 *>(vc + src + i * kAt * D));
                ks[e] = __ldcg(a.k_scales + (piece >> bs16_log2));
                vs[e] = __ldcg(a.v_scales + (piece >> bs16_log2));
            };
            // codes x of step j to `half` of the memory
            auto widen = [&](const uint4 (&x)[kLoads], int j, unsigned char *half) {
                const int key0 = (at.j + j) * kKeys + w * 16 + row0;  // of the sequence
                const bool cut = key0 - row0 + 16 > L;
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    uint4 c = x[i];
                    // rows that hold no token may hold anything
                    if (cut && key0 + i * kAt >= L) c = make_uint4(0, 0, 0, 0);
                    unsigned char *dst = half + (i * kAt & ~7) * 128;
                    *reinterpret_cast<uint4 *>(dst + to[kAt == 8 ? 0 : i & 1][0]) =
                        make_uint4(q8_widen<KIND, 0>(c.x), q8_widen<KIND, 1>(c.x), q8_widen<KIND, 0>(c.y),
                                   q8_widen<KIND, 1>(c.y));
                    *reinterpret_cast<uint4 *>(dst + to[kAt == 8 ? 0 : i & 1][1]) =
                        make_uint4(q8_widen<KIND, 0>(c.z), q8_widen<KIND, 1>(c.z), q8_widen<KIND, 0>(c.w),
                                   q8_widen<KIND, 1>(c.w));
                }
            };
            load(0, 0);
            load(1, 1);
#pragma unroll 1
            for (int j0 = 0; j0 < n && ok; j0 += 2) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = j0 + e, kf = f + j, s = kf % kStages;
                    if (j >= n || !ok) break;
                    ok = warp_wait_or_stop(&sh.empty[s], ((kf / kStages) & 1) ^ 1, stop);
                    if (!ok) break;
                    if (lane == 0) {  // keys behind the sequence have no scale of their own
                        const bool some = (at.j + j) * kKeys + w * 16 < L;
                        sh.f[s][w] = some ? fmaxf(ks[e] * scale, 1e-30f) : 1e-30f;
                        sh.v[s][w] = some ? vs[e] : 0.f;
                    }
                    widen(xk[e], j, ring + 2 * s * C::kHalf);
                    widen(xv[e], j, ring + (2 * s + 1) * C::kHalf);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.full[s]);
                    load(e, j + 2);
                }
            }
            f += n;
        }
    } else {
        // --- softmax, results ---
        const int w = warp >> 2;  // the tile
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 * (warp % 4) << 16
        const uint32_t ts = tmem + 128 * w + lanes, to = tmem + 256 + 128 * w + lanes;
        unsigned char *ws = static_cast<unsigned char *>(a.workspace);
        // records: float4 [D / 4][record_rows], then reference and sum of each row
        auto record_of = [&](int of_cta, int side) {
            return reinterpret_cast<float4 *>(ws + kBalancedCounterBytes) +
                   (2ll * of_cta + side) * (D / 4 + 1) * a.record_rows;
        };
        int shares = 0;
        int f = 0, sc = 0;
        bool ok = true;
#pragma unroll 1
        for (int u = U0; u < U1; at.next(t, a)) {
            int first = u - at.j, n = min(at.steps - at.j, U1 - u);
            int mine = max(0, min(at.steps_of_tile(t, a, w) - at.j, n));
            u += n;
            int left = Place::keys(t, at.b, 2 * at.p * a.tile_tokens + Row(a, threadIdx.x).tok) - at.j * kKeys;
            volatile Piece *keep = &sh.keep[warp];
            if (lane == 0) {
                keep->u = u;
                keep->first = first;
                keep->n = n;
                keep->f = f;
                keep->mine = mine;
                keep->shares = shares;
                keep->b = at.b;
                keep->h = at.h;
                keep->p = at.p;
                keep->steps = at.steps;
            }
            int slot = f % kStages;
            bool fresh = true;
            float r = 0.f, l = 0.f, wv = 0.f, inv_w = 0.f;
#pragma unroll 1
            for (; ok && mine > 0; --mine, ++sc, left -= kKeys, slot = (slot + 1) % kStages) {
                const uint32_t here = ts + 64 * (sc & 1);
                ok = warp_wait_or_stop(&sh.s_full[w][sc & 1], (sc >> 1) & 1, stop);
                if (!ok) break;
                tc_fence_after();
                uint32_t x[2][32];
                tmem_ld32(x[0], here);
                tmem_ld32(x[1], here + 32);
                const float *fg = sh.f[slot], *vg = sh.v[slot];
                float most = kQ8LeastReference;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) most = fmaxf(most, vg[g]);
                tmem_wait_ld();
                if (a.scale_log2 < 0.f)
#pragma unroll
                    for (int c = 0; c < 64; ++c) x[c / 32][c % 32] ^= 0x80000000u;
                if (__any_sync(~0u, left < kKeys))
#pragma unroll
                    for (int c = 0; c < 64; ++c) x[c / 32][c % 32] = c < left ? x[c / 32][c % 32] : 0xff800000u;
                // --- references
                float top = -INFINITY;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const uint32_t *z = &x[g / 2][g % 2 * 16];
                    float m0 = __uint_as_float(z[0]), m1 = __uint_as_float(z[1]);
#pragma unroll
                    for (int c = 2; c + 3 < 16; c += 4) {
                        m0 = max3(m0, __uint_as_float(z[c]), __uint_as_float(z[c + 1]));
                        m1 = max3(m1, __uint_as_float(z[c + 2]), __uint_as_float(z[c + 3]));
                    }
                    m0 = max3(m0, __uint_as_float(z[14]), __uint_as_float(z[15]));
                    top = fmaxf(top, fmaxf(m0, m1) * fg[g]);
                }
                const bool far = !(most >= wv * (1.f / 64.f) && most <= wv * 16.f);
                float fac = 1.f;
                if (far) {
                    inv_w = __fdividef(1.f, most);
                    fac = wv * inv_w;
                    wv = most;
                }
                if (fresh) {
                    fresh = false;
                    r = top > -INFINITY ? top : 0.f;
                } else {
                    const bool move = top - r > kLag;
                    if (__any_sync(~0u, move || far)) {
                        const float next = move ? top : r, g = ex2(r - next);
                        r = next;
                        l *= g;
                        fac *= g;
                        // the outputs so far
                        ok = warp_wait_or_stop(&sh.pv_done[w][(sc - 1) & 1], ((sc - 1) >> 1) & 1, stop);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(o, to + c);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fac);
                            tmem_st16(to + c, o);
                        }
                    }
                }
                // --- weights
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t p[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const int g = 2 * half + c / 8;
                        const float fc = fg[g], v = vg[g] * inv_w;
                        const uint32_t *z = &x[half][2 * c];
                        const float2 e = fma2(make_float2(__uint_as_float(z[0]), __uint_as_float(z[1])), fc, -r);
                        const float2 y = make_float2(ex2(e.x), ex2(e.y));
                        sum = add2(sum, y);
                        const float2 m = mul2(y, make_float2(v, v));
                        p[c] = pack_half2(m.x, m.y);
                    }
                    tmem_st16(here + 16 * half, p);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_ready[w][sc & 1]);
                l += sum.x + sum.y;
            }
            __syncwarp();
            u = keep->u;
            first = keep->first;
            n = keep->n;
            f = keep->f + n;
            mine = keep->mine;
            shares = keep->shares;
            at.b = keep->b;
            at.h = keep->h;
            at.p = keep->p;
            at.steps = keep->steps;
            int tid;
            asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
            const Row row(a, tid);
            const int tokens = start[at.b + 1] - start[at.b] - 2 * at.p * a.tile_tokens;  // from the pair on
            if (ok && mine > 0) {
                ok = warp_wait_or_stop(&sh.pv_done[w][(sc - 1) & 1], ((sc - 1) >> 1) & 1, stop);
                tc_fence_after();
            }
            // after a wait that gave up results are unspecified, but each arrival is made
            if (!ok) mine = 0;
            const bool whole = first >= U0 && first + at.steps <= U1, valid = row.tok < tokens;
            const float inv = wv / l;
            uint4 *out = reinterpret_cast<uint4 *>(static_cast<__half *>(a.out) + row.out_row(t, a, at.b, at.h, at.p) * D);
            float4 *rec = record_of(cta, first >= U0) + row.in_pair;
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                if (mine > 0) {
                    tmem_ld32(o, to + c);
                    tmem_wait_ld();
                    if (c + 32 == D) {  // the next piece's products may write O
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.o_free[w]);
                    }
                }
                if (valid && whole) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t z[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            z[k] = pack_half2(__uint_as_float(o[8 * e + 2 * k]) * inv,
                                              __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                        out[c / 8 + e] = make_uint4(z[0], z[1], z[2], z[3]);
                    }
                } else if (valid) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        __stcg(rec + (c / 4 + e) * a.record_rows,
                               mine > 0 ? make_float4(__uint_as_float(o[4 * e]) * wv, __uint_as_float(o[4 * e + 1]) * wv,
                                                      __uint_as_float(o[4 * e + 2]) * wv,
                                                      __uint_as_float(o[4 * e + 3]) * wv)
                                        : make_float4(0.f, 0.f, 0.f, 0.f));
                }
                __syncwarp();  // the next load is the whole warp's
            }
            if (whole) {
                if (a.lse_out && valid)
                    a.lse_out[row.out_row(t, a, at.b, at.h, at.p)] = (r + log2f(l)) * kLn2;
                continue;
            }
            if (!__any_sync(~0u, valid)) continue;
            if (valid)
                __stcg(rec + (D / 4) * a.record_rows,
                       make_float4(mine > 0 && l != 0.f ? r : -INFINITY, mine > 0 ? l : 0.f, 0.f, 0.f));
            __syncwarp();
            const int from = ranges.of(first);
            if (lane == 0)
                sh.todo[warp][shares] = Share{
                    at.b, at.h, at.p, from, ranges.of(first + at.steps - 1) - from + 1,
                    atomic_add_acq_rel_gpu(reinterpret_cast<int *>(ws) + from * 8 + warp, 1)};
            ++shares;
        }
        // --- joins, by the last warp to arrive with these rows
        const Row row(a, threadIdx.x);
#pragma unroll 1
        for (int i = 0; i < shares; ++i) {
            __syncwarp();
            const Share of = sh.todo[warp][i];
            int last = 0;
            if (lane == 0) {
                int *counter = reinterpret_cast<int *>(ws) + of.from * 8 + warp;
                if (counter_not_zeroed(of.before, of.parts - 1)) {
                    flag_error(a.err, PKV_ERRBIT_WORKSPACE);
                    atomic_exch_relaxed_gpu(counter, kCounterPoison);
                } else if (of.before == of.parts - 1) {
                    last = 1;
                    red_add_relaxed_gpu(counter, -of.parts);
                }
            }
            if (!__shfl_sync(~0u, last, 0)) continue;
            if (row.tok >= start[of.b + 1] - start[of.b] - 2 * of.p * a.tile_tokens) continue;
            float high = -INFINITY;
#pragma unroll 1
            for (int k = 0; k < of.parts; ++k)
                high = fmaxf(high, __ldcg(&(record_of(of.from + k, k == 0) + (D / 4) * a.record_rows + row.in_pair)->x));
            if (high == -INFINITY) high = 0.f;
            const long long out_row = row.out_row(t, a, of.b, of.h, of.p);
            float sum = 0.f;
#pragma unroll 1
            for (int c0 = 0; c0 < D / 4; c0 += 8) {
                float4 acc[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                sum = 0.f;
#pragma unroll 1
                for (int k0 = 0; k0 < of.parts; k0 += 2) {  // the loads of two parts go out together
                    float4 z[2][8];
                    float2 ml[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float4 *part = record_of(of.from + min(k0 + k, of.parts - 1), k0 + k == 0) + row.in_pair;
#pragma unroll
                        for (int e = 0; e < 8; ++e) z[k][e] = __ldcg(part + (c0 + e) * a.record_rows);
                        ml[k] = __ldcg(reinterpret_cast<const float2 *>(part + (D / 4) * a.record_rows));
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (k0 + k >= of.parts) continue;
                        const float g = ex2(ml[k].x - high);
                        sum += g * ml[k].y;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            acc[e].x += g * z[k][e].x;
                            acc[e].y += g * z[k][e].y;
                            acc[e].z += g * z[k][e].z;
                            acc[e].w += g * z[k][e].w;
                        }
                    }
                }
                const float inv = 1.f / sum;
                uint4 *out = reinterpret_cast<uint4 *>(static_cast<__half *>(a.out) + out_row * D) + c0 / 2;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    out[e] = make_uint4(pack_half2(acc[2 * e].x * inv, acc[2 * e].y * inv),
                                        pack_half2(acc[2 * e].z * inv, acc[2 * e].w * inv),
                                        pack_half2(acc[2 * e + 1].x * inv, acc[2 * e + 1].y * inv),
                                        pack_half2(acc[2 * e + 1].z * inv, acc[2 * e + 1].w * inv));
            }
            if (a.lse_out) a.lse_out[out_row] = (high + log2f(sum)) * kLn2;
        }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && sh.stop) {
        flag_error(a.err, PKV_ERRBIT_TIMEOUT);
        // every copy in flight lands before the CTA gives its memory back
        for (int w = 0; w < 2; ++w)
            if (sh.queries[w] > 0) mbar_wait_bounded(&sh.q_full[w], (sh.queries[w] - 1) & 1);
    }
    __syncwarp();
    if (warp == 12) tmem_free(tmem, 512);
}

template <int KIND, int D>
cudaError_t launch(const Q8AttentionArgs &a, const Q8Split &sp, cudaStream_t stream) {
    auto kern = q8_prefill_kernel<KIND, D>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(kern, static_cast<int>(Cfg<D>::smem(kQ8MaxSeqs)), done);
    if (e != cudaSuccess) return e;
    CUtensorMap q_map;
    auto fn = encode_fn();
    const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(a.n_q_heads), static_cast<cuuint64_t>(a.total_q)};
    const cuuint64_t strides[2] = {D * 2, static_cast<cuuint64_t>(a.q_stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.n_q_heads / a.n_kv_heads),
                               static_cast<cuuint32_t>(a.tile_tokens)};
    const cuuint32_t one[3] = {1, 1, 1};
    if (!fn) return cudaErrorNotSupported;
    if (fn(&q_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(a.q), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;  // a stride that the map does not take
    return launch_pdl(kern, dim3(sp.ctas), dim3(kThreads), Cfg<D>::smem(a.num_seqs), stream, a, q_map);
}

static_assert(Cfg<128>::smem(kQ8MaxSeqs) <= 227 * 1024 - 2048, "shared memory");

}  // namespace

bool q8_prefill_fits(int num_seqs, int max_q_len, int n_q_heads, int n_kv_heads, int max_len) {
    if (max_len > kMaxTokens) return false;
    const int tile_tokens = kRows / (n_q_heads / n_kv_heads);
    const double steps = (static_cast<double>(max_len) + kKeys - 1) / kKeys + 1;
    const double pairs = static_cast<double>(max_q_len) / (2 * tile_tokens) + 1;
    return static_cast<double>(num_seqs) * n_kv_heads * pairs * steps <= kQ8MaxUnits;
}

// q8_split for the kernel of this file.
Q8Split q8_prefill_split(int max_q_len, int n_q_heads, int n_kv_heads, int head_dim, int sms) {
    const int group = n_q_heads / n_kv_heads;
    Q8Split sp{};
    sp.tile_tokens = kRows / group;
    sp.ctas = sms < kBalancedMaxWorkers / 8 ? sms : kBalancedMaxWorkers / 8;  // a counter for each warp of rows
    // rows of a pair that may be some: those of one tile, or of both
    sp.record_rows = max_q_len > sp.tile_tokens ? kPair : (max_q_len * group + 31) / 32 * 32;
    sp.ws_bytes = kBalancedCounterBytes +
                  static_cast<size_t>(sp.ctas) * 2 * (head_dim / 4 + 1) * sp.record_rows * sizeof(float4);
    return sp;
}

cudaError_t launch_q8_prefill(const Q8AttentionArgs &a, int kind, const Q8Split &sp, cudaStream_t stream) {
    if (a.head_dim == 128)
        return kind == PKV_Q8_E4M3 ? launch<PKV_Q8_E4M3, 128>(a, sp, stream)
                                   : launch<PKV_Q8_INT8, 128>(a, sp, stream);
    return kind == PKV_Q8_E4M3 ? launch<PKV_Q8_E4M3, 64>(a, sp, stream) : launch<PKV_Q8_INT8, 64>(a, sp, stream);
}

}  // namespace pkv
