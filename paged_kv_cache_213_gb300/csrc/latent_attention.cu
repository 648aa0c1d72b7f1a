// latent_attention.cu -- absorbed latent attention over the paged cache
// (paged_latent_attention): an even split of the batch's work over one CTA per
// SM, and the join of the pieces.
//
// A cache row of E = R + 64 fp16 values is the key of every head, its first R
// values the value, so a tile of tokens is read once and used by all N query
// rows (head x token of one sequence) of a row tile:
//   S^T [64 tokens x N] = K [64 x E] Q^T          (tcgen05, M = 64)
//   P^T = 2^(S^T scale - r), r a reference per row (the softmax warps)
//   O^T [R x N] += V^T [R x 64] P^T               (tcgen05, R / 128 tiles of M = 128)
// Tokens are the M side of the first product and the value columns that of the
// second: with few rows (N = 16 .. 64) no tensor-core row is padding, O^T takes
// only N TMEM columns a tile, and both operands of the second product are the
// bytes already in shared memory, read along their other axis.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <cmath>
#include <mutex>

#include "pagedkv_latent.h"
#include "pkv_internal.h"
#include "rope_latent.h"
#include "tc05.cuh"

namespace pkv {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

namespace {

constexpr int kTile = 64;      // tokens
constexpr int kThreads = 192;  // softmax warps 0-3, copy warp 4, MMA warp 5
// P holds 2^(s - r) with r kHead below the running maximum: weights up to
// 2^kHead, and up to 2^(kHead + kLag) before r follows; fp16 ends at 2^16.
constexpr float kHead = 6.f, kLag = 8.f;

template <int R, int N>
struct Cfg {
    static constexpr int E = R + 64, PL = E / 64, VT = R / 128;
    static constexpr int PLANE = kTile * 128, QPLANE = N * 128;
    static constexpr int STAGE = PL * PLANE;
    static constexpr int STAGES = R == 512 ? 2 : 4;
    static constexpr int Q_BYTES = PL * QPLANE, P_BYTES = kTile * 128;
    static constexpr int SMEM = 1024 + STAGES * STAGE + Q_BYTES + P_BYTES;
    static constexpr int COLS = (VT + 2) * N;
    static constexpr int TMEM = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
};

// One sequence's work: its query rows and how many of its tokens each attends.
struct Seq {
    int q0, n, len;  // first query token, query tokens, cached tokens
};

// False for a sequence out of bounds (no work).  An empty sequence of the
// one-token form keeps its row, which attends nothing.
__device__ __forceinline__ bool load_seq(const LatentAttentionArgs &a, int b, Seq *s) {
    s->q0 = b;
    s->n = 1;
    s->len = a.context_lens[b];
    if (a.query_start) {
        s->q0 = a.query_start[b];
        s->n = a.query_start[b + 1] - s->q0;
    }
    const bool empty = !a.query_start && s->len == 0;
    return s->len >= 0 && s->len <= a.max_context_len && s->n >= 0 && s->n <= a.max_q_len &&
           s->q0 >= 0 && s->n <= a.total_q - s->q0 && (s->n <= s->len || empty);
}

// Tokens that the rows of a row tile attend at most.
__device__ __forceinline__ int tile_end(const Seq &s, int heads, int rows, int rt) {
    const int last = min(static_cast<int>((static_cast<long long>(rt + 1) * rows - 1) / heads), s.n - 1);
    return s.len > 0 ? s.len - s.n + last + 1 : 0;
}

__device__ __forceinline__ int row_tiles(const Seq &s, int heads, int rows) {
    return static_cast<int>((static_cast<long long>(s.n) * heads + rows - 1) / rows);
}

__device__ __forceinline__ int token_tiles(int end) {
    return end > 0 ? (end + kTile - 1) / kTile : 1;
}

// Units (token tiles) of a whole sequence.
__device__ __forceinline__ long long seq_units(const LatentAttentionArgs &a, int b, int rows,
                                               bool *good) {
    Seq s;
    *good = load_seq(a, b, &s);
    if (!*good || s.n == 0) return 0;
    if (s.n == 1) return static_cast<long long>(row_tiles(s, a.n_q_heads, rows)) * token_tiles(s.len);
    long long u = 0;
    for (int rt = row_tiles(s, a.n_q_heads, rows) - 1; rt >= 0; --rt)
        u += token_tiles(tile_end(s, a.n_q_heads, rows, rt));
    return u;
}

// A CTA's place in the split: units [first, first + left) starting `skip` units
// into sequence `b`.
struct Range {
    int b;
    long long skip, left, first, total;
    int workers;
};

// A run of token tiles of one (sequence, row tile).
struct Piece {
    Seq s;
    int b, rt, t0, tiles, end;  // end: tokens of the whole segment
    int seg_tiles;
    long long seg_first;        // unit at which the segment starts
};

struct Walk {
    int b, rt;
    long long skip, left, unit;
};

__device__ __forceinline__ Walk start_walk(const Range &r) {
    return Walk{r.b, 0, r.skip, r.left, r.first - r.skip};
}

__device__ bool next_piece(const LatentAttentionArgs &a, int rows, Walk *w, Piece *p) {
    if (w->left <= 0) return false;
    while (w->b < a.num_seqs) {
        Seq s;
        if (load_seq(a, w->b, &s)) {
            const int rts = row_tiles(s, a.n_q_heads, rows);
            for (; w->rt < rts; ++w->rt) {
                const int end = tile_end(s, a.n_q_heads, rows, w->rt);
                const int tiles = token_tiles(end);
                if (w->skip >= tiles) {
                    w->skip -= tiles;
                    w->unit += tiles;
                    continue;
                }
                const int t0 = static_cast<int>(w->skip);
                const int take = static_cast<int>(min(static_cast<long long>(tiles - t0), w->left));
                *p = Piece{s, w->b, w->rt, t0, take, end, tiles, w->unit};
                w->left -= take;
                w->skip = 0;
                w->unit += tiles;
                ++w->rt;
                return true;
            }
        }
        ++w->b;
        w->rt = 0;
    }
    return false;
}

// Workspace: a record per CTA {first output row, rows, last CTA of the segment or
// -1, 0}, then per piece slot (two a CTA: 0 ends a segment or lies inside one, 1
// starts one) N pairs (r, l) and N x R partial sums.
struct Layout {
    size_t ml, acc, total;
};

__host__ __device__ inline Layout layout(int workers, int rows, int R) {
    Layout l;
    l.ml = (static_cast<size_t>(workers) * 16 + 255) / 256 * 256;
    l.acc = l.ml + static_cast<size_t>(2 * workers) * rows * 8;
    l.total = l.acc + static_cast<size_t>(2 * workers) * rows * R * 4;
    return l;
}

struct Shared {
    uint64_t full[4], empty[4], s_full[2], p_ready, q_full, q_empty, o_full, o_free, drained;
    uint32_t tmem;
    int stop;
    Range range;
    long long sums[kThreads / 32];
    float warps[4][64];  // per row, of each softmax warp: a tile's maxima, a piece's sums
    float factor[64];    // what O^T's columns are multiplied with
    float ref[64];
};

__device__ __forceinline__ bool any_softmax(bool x) {  // over the four softmax warps
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.aligned.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x))
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void sync_softmax() {
    __syncwarp();
    asm volatile("barrier.cta.sync.aligned 1, 128;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void load_scores(uint32_t (&x)[N / 2], uint32_t addr) {
    if constexpr (N == 64) tmem_ld_m8(x, addr);
    if constexpr (N == 32) tmem_ld_m4(x, addr);
    if constexpr (N == 16) tmem_ld_m2(x, addr);
}

static_assert(sizeof(Shared) <= 2048, "beside the largest configuration's 225 KB");

template <int R, int N>
__global__ void __launch_bounds__(kThreads, 1)
    latent_attention_kernel(const LatentAttentionArgs a, const __grid_constant__ CUtensorMap mq,
                            const __grid_constant__ CUtensorMap mc) {
    using C = Cfg<R, N>;
    extern __shared__ unsigned char raw[];
    __shared__ Shared sh;
    unsigned char *base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    unsigned char *q_smem = base + C::STAGES * C::STAGE, *p_smem = q_smem + C::Q_BYTES;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = a.n_q_heads;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        mbar_init(&sh.s_full[0], 1);
        mbar_init(&sh.s_full[1], 1);
        mbar_init(&sh.p_ready, 4);
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.o_full, 1);
        mbar_init(&sh.o_free, 4);
        mbar_init(&sh.drained, 1);
        sh.stop = 0;
        fence_barrier_init();
    }
    if (warp == 5) {
        tmem_alloc(&sh.tmem, C::TMEM);
        if (lane == 0) {
            prefetch_tmap(&mq);
            prefetch_tmap(&mc);
        }
    }
    grid_dependency_wait();
    allow_dependent_launch();

    // the split: every CTA sums the units of all sequences and finds its range
    {
        const int per = (a.num_seqs + kThreads - 1) / kThreads;
        const int b0 = min(static_cast<int>(threadIdx.x) * per, a.num_seqs);
        const int b1 = min(b0 + per, a.num_seqs);
        long long mine = 0;
        bool good;
        for (int b = b0; b < b1; ++b) {
            mine += seq_units(a, b, N, &good);
            if (!good && blockIdx.x == 0) flag_error(a.err, PKV_ERRBIT_CONTEXT);
        }
        // inclusive scan: within the warp by shuffles, over the warps in shared memory
        long long acc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, acc, o);
            if (lane >= o) acc += v;
        }
        if (lane == 31) sh.sums[warp] = acc;
        if (threadIdx.x == 0) sh.range.left = 0;
        __syncthreads();
        long long before = acc - mine, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += sh.sums[w];
            total += sh.sums[w];
        }
        const int workers = static_cast<int>(min(total, static_cast<long long>(gridDim.x)));
        if (static_cast<int>(blockIdx.x) < workers) {
            const long long first = static_cast<long long>(blockIdx.x) * total / workers;
            const long long last = static_cast<long long>(blockIdx.x + 1) * total / workers;
            if (mine > 0 && before <= first && first < before + mine) {
                int b = b0;
                long long at = before;
                for (; b < b1; ++b) {
                    const long long u = seq_units(a, b, N, &good);
                    if (first < at + u) break;
                    at += u;
                }
                sh.range = Range{b, first - at, last - first, first, total, workers};
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    volatile int *stop = &sh.stop;
    const Range range = sh.range;

    if (range.left <= 0) {
        if (threadIdx.x == 0)
            static_cast<int4 *>(a.workspace)[blockIdx.x] = make_int4(0, 0, -1, 0);
    } else if (warp == 4) {
        // --- copies ---
        Walk w = start_walk(range);
        Piece p;
        const int box = min(a.block_size, kTile), subs = kTile / box;
        int g = 0, k = 0;  // tiles, pieces so far
        bool ok = true;
        while (ok && next_piece(a, N, &w, &p)) {
            if (lane == 0) {
                ok = wait_or_stop(&sh.q_empty, (k & 1) ^ 1, stop);
                if (ok) {
                    mbar_arrive_expect_tx(&sh.q_full, C::Q_BYTES);
                    const int row = p.s.q0 * H + p.rt * N;
                    for (int x = 0; x < C::PL; ++x)
                        tma_load_2d(q_smem + x * C::QPLANE, &mq, 64 * x, row, &sh.q_full);
                }
            }
            ++k;
            const int32_t *table = a.block_tables + static_cast<long long>(p.b) * a.max_blocks_per_seq;
            auto block_of = [&](int t) {  // this lane's block of tile t, or -1
                const int token = t * kTile + lane * box;
                if (lane >= subs || token >= p.s.len || t >= p.t0 + p.tiles) return -1;
                const int id = table[token / a.block_size];
                if (id >= 0 && id < a.num_blocks) return id;
                flag_error(a.err, PKV_ERRBIT_BLOCK_ID);
                return 0;  // some block of the pool: the sequence's result is unspecified
            };
            int id = block_of(p.t0);
            for (int t = p.t0; t < p.t0 + p.tiles; ++t, ++g) {
                const int next = block_of(t + 1);
                const int s = g % C::STAGES;
                if (lane == 0) ok = ok && wait_or_stop(&sh.empty[s], ((g / C::STAGES) & 1) ^ 1, stop);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                const int live = __popc(__ballot_sync(0xffffffffu, id >= 0));
                if (lane == 0) {
                    if (live > 0)
                        mbar_arrive_expect_tx(&sh.full[s], live * box * C::E * 2);
                    else
                        mbar_arrive(&sh.full[s]);
                }
                __syncwarp();
                if (id >= 0) {
                    const int row = id * a.block_size + (t * kTile + lane * box) % a.block_size;
                    unsigned char *dst = base + s * C::STAGE + lane * box * 128;
                    for (int x = 0; x < C::PL; ++x)
                        tma_load_2d(dst + x * C::PLANE, &mc, 64 * x, row, &sh.full[s]);
                }
                id = next;
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        if (!ok && lane == 0) {
            // every copy in flight lands before the CTA gives its memory back
            mbar_wait_bounded(&sh.q_full, (k - 1) & 1);
            for (int i = max(0, g - C::STAGES); i < g; ++i)
                mbar_wait_bounded(&sh.full[i % C::STAGES], (i / C::STAGES) & 1);
        }
    } else if (warp == 5) {
        // --- matrix products ---
        if (elect_one()) {
            constexpr uint32_t ds = mma_desc(kTile, N, false, false);
            constexpr uint32_t dpv = mma_desc(128, N, true, true);
            const uint32_t kv = smem_addr(base), qa = smem_addr(q_smem), pa = smem_addr(p_smem);
            Walk w = start_walk(range);
            Piece p;
            int g = 0, k = 0;
            bool ok = true;
            while (ok && next_piece(a, N, &w, &p)) {
                ok = wait_or_stop(&sh.q_full, k & 1, stop);
                int sj = 0, pj = 0;
                unsigned spins = 0;
                unsigned long long t0 = 0;
                while (ok && pj < p.tiles) {
                    const int gs = g + sj, gp = g + pj;
                    if (sj < p.tiles && sj < pj + 2 &&
                        mbar_test_wait(&sh.full[gs % C::STAGES], (gs / C::STAGES) & 1)) {
                        const uint32_t ka = kv + (gs % C::STAGES) * C::STAGE;
                        const uint32_t d = tmem + (C::VT + (gs & 1)) * N;
                        tc_fence_after();
#pragma unroll
                        for (int x = 0; x < 4 * C::PL; ++x)
                            mma_ss(d, smem_desc(ka + (x / 4) * C::PLANE + (x % 4) * 32, 1024, 0),
                                   smem_desc(qa + (x / 4) * C::QPLANE + (x % 4) * 32, 1024, 0), ds,
                                   x > 0);
                        mma_commit(&sh.s_full[gs & 1]);
                        if (++sj == p.tiles) mma_commit(&sh.q_empty);
                        spins = 0;
                    } else if (pj < sj && mbar_test_wait(&sh.p_ready, gp & 1)) {
                        if (pj == 0) {
                            ok = wait_or_stop(&sh.o_free, (k & 1) ^ 1, stop);
                            if (!ok) break;
                        }
                        const uint32_t va = kv + (gp % C::STAGES) * C::STAGE;
                        tc_fence_after();
#pragma unroll
                        for (int v = 0; v < C::VT; ++v)
#pragma unroll
                            for (int x = 0; x < kTile / 16; ++x)
                                mma_ss(tmem + v * N,
                                       smem_desc(va + 2 * v * C::PLANE + x * 2048, 1024, C::PLANE),
                                       smem_desc(pa + x * 2048, 1024, 0), dpv, pj > 0 || x > 0);
                        mma_commit(&sh.empty[gp % C::STAGES]);
                        if (++pj == p.tiles) mma_commit(&sh.o_full);
                        spins = 0;
                    } else if ((++spins & 255u) == 0) {
                        if (spins == 256) t0 = global_timer_ns();
                        if (*stop || spins > kWaitLimitIters ||
                            global_timer_ns() - t0 > kWaitLimitNs) {
                            *stop = 1;
                            ok = false;
                        }
                    }
                }
                g += p.tiles;
                ++k;
            }
            // nothing of the tensor core is left in flight when TMEM is freed
            mma_commit(&sh.drained);
            mbar_wait_bounded(&sh.drained, 0);
        }
    } else {
        // --- softmax, results ---
        // scores: this thread holds tokens 16 warp + lane / 4 (+ 8) and rows
        // 8 c + 2 (lane % 4) (+ 1), c < N / 8
        constexpr int NC = N / 8;
        const uint32_t lanes = static_cast<uint32_t>(warp) << 21;
        const int tok = 16 * warp + lane / 4, col = 2 * (lane & 3);
        const Layout lay = layout(gridDim.x, N, R);
        char *ws = static_cast<char *>(a.workspace);
        const float scale = a.scale_log2;
        Walk w = start_walk(range);
        Piece p;
        int g = 0, k = 0;
        bool recorded = false;
        while (next_piece(a, N, &w, &p)) {
            float ref[NC][2], sum[NC][2];
            int seen[NC][2];  // tokens that the row attends
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = (p.rt * N + 8 * c + col + e) / H;
                    seen[c][e] = p.s.n == 1 ? p.s.len : min(p.s.len - p.s.n + i + 1, p.s.len);
                    ref[c][e] = sum[c][e] = 0.f;
                }
            // tiles below this one need no mask
            const int first_masked =
                (p.s.n == 1 ? p.s.len : p.s.len - p.s.n + (p.rt * N) / H + 1) / kTile;
            for (int j = 0; j < p.tiles; ++j, ++g) {
                const int t = p.t0 + j;
                warp_wait_or_stop(&sh.s_full[g & 1], (g >> 1) & 1, stop);
                tc_fence_after();
                uint32_t xr[N / 2];
                load_scores<N>(xr, tmem + (C::VT + (g & 1)) * N + lanes);
                tmem_wait_ld();
                float x[NC][4];  // [c][2 * (second token) + (second row)]
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[c][e] = __uint_as_float(xr[4 * c + e]);
                        if (a.negate) x[c][e] = -x[c][e];
                    }
                if (t >= first_masked) {
                    const int at = t * kTile + tok;
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (at + 8 * (e >> 1) >= seen[c][e & 1]) x[c][e] = -INFINITY;
                }
                float top[NC][2];
                bool move = j == 0;
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        top[c][e] = fmaxf(x[c][e], x[c][2 + e]) * scale;
                        move |= top[c][e] - ref[c][e] > kHead + kLag;
                    }
                if (any_softmax(move)) {
                    // new references: the tile's maxima over all tokens
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1)
                                top[c][e] = fmaxf(top[c][e], __shfl_xor_sync(0xffffffffu, top[c][e], o));
                            if (lane < 4) sh.warps[warp][8 * c + col + e] = top[c][e];
                        }
                    sync_softmax();
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int n = 8 * c + col + e;
                            const float m = fmaxf(fmaxf(sh.warps[0][n], sh.warps[1][n]),
                                                  fmaxf(sh.warps[2][n], sh.warps[3][n]));
                            float next = ref[c][e];
                            if (j == 0)
                                next = m > -INFINITY ? m - kHead : 0.f;
                            else if (m - next > kHead + kLag)
                                next = m - kHead;
                            const float f = j == 0 ? 1.f : ex2(ref[c][e] - next);
                            sum[c][e] *= f;
                            ref[c][e] = next;
                            if (warp == 0 && lane < 4) sh.factor[n] = f;
                        }
                    sync_softmax();
                    if (j > 0) {
                        // O^T's columns follow, after the products into it
                        warp_wait_or_stop(&sh.empty[(g - 1) % C::STAGES],
                                          ((g - 1) / C::STAGES) & 1, stop);
                        tc_fence_after();
#pragma unroll 1
                        for (int v = 0; v < C::VT * N; v += 16) {
                            uint32_t o[16];
                            tmem_ld16(o, tmem + v + lanes);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) *
                                                       sh.factor[v % N + e]);
                            tmem_st16(tmem + v + lanes, o);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                }
                uint32_t y[NC][2];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float p0 = ex2(fmaf(x[c][0], scale, -ref[c][0]));
                    const float p1 = ex2(fmaf(x[c][1], scale, -ref[c][1]));
                    const float p2 = ex2(fmaf(x[c][2], scale, -ref[c][0]));
                    const float p3 = ex2(fmaf(x[c][3], scale, -ref[c][1]));
                    sum[c][0] += p0 + p2;
                    sum[c][1] += p1 + p3;
                    y[c][0] = pack_half2(p0, p1);
                    y[c][1] = pack_half2(p2, p3);
                }
                // the one P buffer is free when the products before are done
                if (g > 0)
                    warp_wait_or_stop(&sh.empty[(g - 1) % C::STAGES], ((g - 1) / C::STAGES) & 1,
                                      stop);
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = tok + 8 * e;
                        *reinterpret_cast<uint32_t *>(p_smem + r * 128 + ((c ^ (r & 7)) << 4) +
                                                      2 * col) = y[c][e];
                    }
                // values of rows past the sequence's end meet weights of 0: they must
                // be finite
                const int valid = p.s.len - t * kTile;
                if (valid < kTile) {
                    unsigned char *v = base + (g % C::STAGES) * C::STAGE;
                    const int pieces = (kTile - valid) * 8;
                    for (int e = threadIdx.x; e < pieces * (R / 64); e += 128)
                        *reinterpret_cast<uint4 *>(v + (e / pieces) * C::PLANE + valid * 128 +
                                                   (e % pieces) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_ready);
            }
            // the row sums, over the tokens of all threads
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1)
                        sum[c][e] += __shfl_xor_sync(0xffffffffu, sum[c][e], o);
                    if (lane < 4) sh.warps[warp][8 * c + col + e] = sum[c][e];
                    if (warp == 0 && lane < 4) sh.ref[8 * c + col + e] = ref[c][e];
                }
            warp_wait_or_stop(&sh.o_full, k & 1, stop);
            tc_fence_after();
            sync_softmax();
            const int rows = min(N, p.s.n * H - p.rt * N);
            const long long row0 = static_cast<long long>(p.s.q0) * H + p.rt * N;
            const bool whole = p.t0 == 0 && p.tiles == p.seg_tiles;
            const int slot = 2 * blockIdx.x + (p.t0 == 0 ? 1 : 0);
            if (threadIdx.x < rows) {
                const int n = threadIdx.x;
                const float l = (sh.warps[0][n] + sh.warps[1][n]) + (sh.warps[2][n] + sh.warps[3][n]);
                if (whole) {
                    sh.factor[n] = l > 0.f || l != l ? 1.f / l : 0.f;
                    if (a.lse_out)
                        a.lse_out[row0 + n] =
                            l == 0.f ? -INFINITY : (sh.ref[n] + log2f(l)) * 0.69314718055994531f;
                } else {
                    reinterpret_cast<float2 *>(ws + lay.ml)[slot * N + n] =
                        make_float2(l == 0.f ? -INFINITY : sh.ref[n], l);
                }
            }
            if (whole) sync_softmax();
            float *acc = reinterpret_cast<float *>(ws + lay.acc) + static_cast<size_t>(slot) * N * R;
            __half *out = static_cast<__half *>(a.out) + row0 * R;
#pragma unroll 1
            for (int v = 0; v < C::VT * N; v += 16) {
                uint32_t o[16];
                tmem_ld16(o, tmem + v + lanes);
                tmem_wait_ld();
                const int d = 128 * (v / N) + 32 * warp + lane;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int n = v % N + e;
                    if (n >= rows) continue;
                    const float f = __uint_as_float(o[e]);
                    if (whole)
                        out[static_cast<size_t>(n) * R + d] = __float2half_rn(f * sh.factor[n]);
                    else
                        acc[static_cast<size_t>(n) * R + d] = f;
                }
            }
            tc_fence_before();
            sync_softmax();  // sh.warps, sh.ref and sh.factor are free again
            if (lane == 0) mbar_arrive(&sh.o_free);
            if (!whole && p.t0 == 0 && threadIdx.x == 0) {
                // this CTA starts the segment: the join finds its last piece here
                const long long last = p.seg_first + p.seg_tiles;
                const int c1 = static_cast<int>((last * range.workers - 1) / range.total);
                static_cast<int4 *>(a.workspace)[blockIdx.x] =
                    make_int4(static_cast<int>(row0), rows, c1, 0);
            }
            recorded |= !whole && p.t0 == 0;
            ++k;
        }
        if (!recorded && threadIdx.x == 0)
            static_cast<int4 *>(a.workspace)[blockIdx.x] = make_int4(0, 0, -1, 0);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sh.stop) flag_error(a.err, PKV_ERRBIT_TIMEOUT);
    __syncwarp();
    if (warp == 5) tmem_free(tmem, C::TMEM);
}

// The pieces of each cut segment, joined: record blockIdx.x, rows blockIdx.y,
// + gridDim.y, ...  Two halves of the block take every other piece.
template <int R>
__global__ void __launch_bounds__(R / 2)
    latent_join_kernel(const LatentAttentionArgs a, int workers, int N) {
    grid_dependency_wait();
    allow_dependent_launch();
    constexpr int T = R / 4;  // threads of one half, 4 columns each
    __shared__ float4 other[T];
    const int4 rec = static_cast<const int4 *>(a.workspace)[blockIdx.x];
    if (rec.z < 0) return;
    const Layout lay = layout(workers, N, R);
    const char *ws = static_cast<const char *>(a.workspace);
    const float2 *ml = reinterpret_cast<const float2 *>(ws + lay.ml);
    const float4 *acc = reinterpret_cast<const float4 *>(ws + lay.acc);
    const int pieces = rec.z - static_cast<int>(blockIdx.x) + 1;
    const int half = threadIdx.x / T, x = threadIdx.x % T, lane = threadIdx.x & 31;
    auto slot = [&](int k) { return 2 * (static_cast<int>(blockIdx.x) + k) + (k == 0 ? 1 : 0); };
    for (int n = blockIdx.y; n < rec.y; n += gridDim.y) {
        float m = -INFINITY;
        for (int k = lane; k < pieces; k += 32) m = fmaxf(m, ml[slot(k) * N + n].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float m0 = m > -INFINITY ? m : 0.f;
        float l = 0.f;
        for (int k = lane; k < pieces; k += 32) {
            const float2 v = ml[slot(k) * N + n];
            l += v.y * ex2(v.x - m0);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = half; k < pieces; k += 2) {
            const size_t at = static_cast<size_t>(slot(k)) * N + n;
            const float f = ex2(ml[at].x - m0);
            const float4 v = acc[at * (R / 4) + x];
            s.x = fmaf(v.x, f, s.x);
            s.y = fmaf(v.y, f, s.y);
            s.z = fmaf(v.z, f, s.z);
            s.w = fmaf(v.w, f, s.w);
        }
        if (half == 1) other[x] = s;
        __syncthreads();
        if (half == 0) {
            const float4 v = other[x];
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            const size_t row = static_cast<size_t>(rec.x) + n;
            reinterpret_cast<uint2 *>(a.out)[row * (R / 4) + x] =
                make_uint2(pack_half2((s.x + v.x) * inv, (s.y + v.y) * inv),
                           pack_half2((s.z + v.z) * inv, (s.w + v.w) * inv));
            if (a.lse_out && x == 0)
                a.lse_out[row] = l == 0.f ? -INFINITY : (m0 + log2f(l)) * 0.69314718055994531f;
        }
        __syncthreads();
    }
}

bool make_map(CUtensorMap *m, const void *base, cuuint64_t rows, cuuint64_t width,
              cuuint32_t box_rows) {
    auto fn = encode_fn();
    const cuuint64_t dims[2] = {width, rows}, strides[1] = {width * 2};
    const cuuint32_t box[2] = {64, box_rows}, one[2] = {1, 1};
    return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void *>(base), dims, strides,
                    box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a row tile: the smallest of 16, 32 and 64 that holds a sequence's rows.
int tile_rows(int max_q_len, int heads) {
    const long long rows = static_cast<long long>(max_q_len) * heads;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

template <int R, int N>
cudaError_t launch(const LatentAttentionArgs &a, int workers, cudaStream_t stream) {
    using C = Cfg<R, N>;
    CUtensorMap mq, mc;
    if (!make_map(&mq, a.q, static_cast<cuuint64_t>(a.total_q) * a.n_q_heads, C::E, N) ||
        !make_map(&mc, a.cache, static_cast<cuuint64_t>(a.num_blocks) * a.block_size, C::E,
                  a.block_size < kTile ? a.block_size : kTile))
        return cudaErrorNotSupported;
    auto kern = latent_attention_kernel<R, N>;
    static std::once_flag once;
    static cudaError_t attr = cudaSuccess;
    std::call_once(once, [&] {
        attr = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (attr != cudaSuccess) return attr;
    cudaError_t e = launch_pdl(kern, dim3(workers), dim3(kThreads), C::SMEM, stream, a, mq, mc);
    if (e != cudaSuccess) return e;
    return launch_pdl(latent_join_kernel<R>, dim3(workers, 16), dim3(R / 2), 0, stream, a, workers, N);
}

}  // namespace

size_t latent_workspace(int max_q_len, int heads, int latent_dim, int workers) {
    return layout(workers, tile_rows(max_q_len, heads), latent_dim).total;
}

cudaError_t launch_latent_attention(const LatentAttentionArgs &a, int workers,
                                    cudaStream_t stream) {
    const int rows = tile_rows(a.max_q_len, a.n_q_heads);
    if (a.latent_dim == 512)
        return rows == 16   ? launch<512, 16>(a, workers, stream)
               : rows == 32 ? launch<512, 32>(a, workers, stream)
                            : launch<512, 64>(a, workers, stream);
    return rows == 16   ? launch<256, 16>(a, workers, stream)
           : rows == 32 ? launch<256, 32>(a, workers, stream)
                        : launch<256, 64>(a, workers, stream);
}

}  // namespace pkv
