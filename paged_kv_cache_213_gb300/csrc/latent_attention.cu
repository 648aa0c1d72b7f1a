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
// bytes already in shared memory, read along their other axis.  Above 64 rows two
// CTAs have 64 each; each copies every tile, the second one's from L2.
//
// A token's row is 1152 bytes at R = 512 and costs 2 (R + E) flops a row: with 128
// rows the copy rate and the product rate of the SMs meet.  What bounds the kernel:
//  few rows    the copies: 32 sequences of 128 .. 2048 tokens x 16 rows 18.5 us, of
//              which 6 are the bytes at the copy rate and the rest the start (every
//              SM's first tiles at once, 4 us), one tile's chain and the join; 64 of
//              1000 .. 3000 35.4 us, 4.2 TB/s;
//  64 rows     two tiles in flight: Q and a tile take 74 KB of shared memory each, and
//              a tile lives about 5500 cycles (copy 1100 .. 1800, scores 1200, softmax
//              1200, products 1000, release 700) for 1870 cycles of products, of which
//              the scores' 1150 are the reads of their operands (4 KB for 16 cycles of
//              arithmetic).  64 sequences of 3000 .. 5000 tokens x 128 rows: 95 us,
//              3.3 TB/s, 750 TFLOP/s.
// P^T is fp16 because the other operand of its product, the cached value, is: half a
// step of each weight, 2^-11, as much as the result's own rounding.  The row sums take
// the weights before that rounding; they, the references and O^T are fp32, in the pieces
// and in the join too.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <atomic>
#include <climits>
#include <cmath>

#include "pagedkv_latent.h"
#include "pkv_internal.h"
#include "rope_latent.h"
#include "tc05.cuh"

namespace pkv {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

namespace {

constexpr int kTile = 64;  // tokens
constexpr int kAhead = 2;  // tiles that the copies into L2 run ahead of those into shared memory
// P holds 2^(s - r) with r kHead below the running maximum: weights up to
// 2^kHead, and up to 2^(kHead + kLag) before r follows; fp16 ends at 2^16.
constexpr float kHead = 6.f, kLag = 8.f;

// CL: CTAs of a worker, which go through the same token tiles with N query rows each.
template <int R, int N, int CL>
struct Cfg {
    static constexpr int E = R + 64, PL = E / 64, VT = R / 128;
    static constexpr int ROWS = CL * N;  // query rows of a worker's row tile
    // A tile comes and goes in parts of PP 64-column planes, each with barriers of its
    // own: the scores start on the first part while the others are on their way, and
    // the next tile's first part follows once the products that read this one's are
    // done.  In shared memory a part is 8 groups of 8 tokens, a group PP planes of
    // 1024 bytes (what one 4-D copy of a block's rows writes).
    static constexpr int PARTS = PL % 3 == 0 ? 3 : 1, PP = PL / PARTS;
    static constexpr int GROUP = PP * 1024, PART = kTile / 8 * GROUP, STAGE = PARTS * PART;
    static constexpr int plane(int x) { return x / PP * PART + x % PP * 1024; }  // its offset
    // the last of the VT output tiles that reads a part (tile v reads planes 2 v and
    // 2 v + 1; the last part holds P^T too)
    static constexpr int last_reader(int part) {
        return part == PARTS - 1 ? VT - 1 : ((part + 1) * PP - 1) / 2;
    }
    static constexpr int STAGES = R == 512 ? 2 : 4;
    static constexpr int Q_GROUP = PL * 1024, Q_BYTES = N / 8 * Q_GROUP;  // groups of all planes
    // P^T takes the place of the tile's last plane (the rotated key part), which
    // nothing reads after the scores: 128 bytes a token
    static constexpr int P_AT = plane(PL - 1);
    static constexpr int SMEM = 1024 + STAGES * STAGE + Q_BYTES;
    static constexpr int COLS = (VT + 2) * N;
    static constexpr int TMEM = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    // softmax warps, four a group; a group takes NG of the rows and VG of O^T's
    // 16-column pieces
    static constexpr int GROUPS = N == 64 ? 2 : 1, SW = 4 * GROUPS;
    static constexpr int NG = N / GROUPS;
    static constexpr int THREADS = 32 * (SW + 3);  // and the copy warp and two for the products
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
    if (s.n == 1) return s.len;
    const int last = min(static_cast<int>((static_cast<unsigned>(rt + 1) * rows - 1) / heads), s.n - 1);
    return s.len - s.n + last + 1;
}

// Row tiles of n query tokens (total_q * heads is at most 2^30).
__device__ __forceinline__ int row_tiles(int n, int heads, int rows) {
    return (n * heads + rows - 1) / rows;
}

__device__ __forceinline__ int token_tiles(int end) {
    return end > 0 ? (end + kTile - 1) / kTile : 1;
}

// Units (token tiles of a row tile) of a whole sequence; the host keeps the sum
// over the batch below 2^31.
__device__ __forceinline__ int seq_units(const Seq &s, int heads, int rows) {
    int u = 0;
    for (int rt = row_tiles(s.n, heads, rows) - 1; rt >= 0; --rt)
        u += token_tiles(tile_end(s, heads, rows, rt));
    return u;
}

// The even split: worker c has the units [first(c), first(c + 1)).
struct Split {
    int each, more;  // units of a worker, workers with one more
    __device__ int first(int c) const { return c * each + min(c, more); }
    __device__ int worker_of(int unit) const {
        const int big = more * (each + 1);
        return unit < big ? unit / (each + 1) : more + (unit - big) / each;
    }
};

// A run of token tiles of one (sequence, row tile).
struct Piece {
    Seq s;
    int b, rt, t0, tiles;
    int seg, seg_tiles, seg_first;  // the segment's number, tiles and first unit
};

// A place in the list of units: `left` units from `skip` units behind the start of
// row tile rt of sequence b, segment `seg` of the batch, which is at `unit`.
struct Walk {
    int b, rt, skip, left, unit, seg;
};

// The piece of sequence w->b (which is s) that w stands at, if there is one.
__device__ __forceinline__ bool piece_of(const Seq &s, int heads, int rows, Walk *w, Piece *p) {
    const int rts = row_tiles(s.n, heads, rows);
    for (; w->rt < rts; ++w->rt) {
        const int tiles = token_tiles(tile_end(s, heads, rows, w->rt));
        if (w->skip >= tiles) {
            w->skip -= tiles;
            w->unit += tiles;
            ++w->seg;
            continue;
        }
        const int take = min(tiles - w->skip, w->left);
        *p = Piece{s, w->b, w->rt, w->skip, take, w->seg, tiles, w->unit};
        w->left -= take;
        w->skip = 0;
        w->unit += tiles;
        ++w->seg;
        ++w->rt;
        return true;
    }
    return false;
}

__device__ __forceinline__ bool next_piece(const LatentAttentionArgs &a, int rows, Walk *w, Piece *p) {
    if (w->left <= 0) return false;
    while (w->b < a.num_seqs) {
        Seq s;
        if (load_seq(a, w->b, &s) && piece_of(s, a.n_q_heads, rows, w, p)) return true;
        ++w->b;
        w->rt = 0;
    }
    return false;
}

// Workspace: `records` x CL records {first output row, rows, first and last worker
// of the segment; no rows: nothing to join}, then per piece slot (two a worker: 0
// ends a segment or lies inside one, 1 starts one) and CTA of the worker N pairs
// (r, l) and N x R partial sums, four rows of a column together, then the columns.
struct Layout {
    size_t ml, acc, total;
};

__host__ __device__ inline Layout layout(int records, int workers, int cl, int rows, int R) {
    const size_t slots = static_cast<size_t>(2 * workers) * cl;
    Layout l;
    l.ml = (static_cast<size_t>(records) * cl * 16 + 255) / 256 * 256;
    l.acc = l.ml + slots * rows * 8;
    l.total = l.acc + slots * rows * R * 4;
    return l;
}

struct Shared {
    uint64_t full[4][3], empty[4][3], s_full[2], p_ready[2], pv_done[2], q_full, q_empty, o_full, o_free, drained[2];
    uint32_t tmem;
    int stop;
    int begun, asked;  // parts of tiles and query copies that were issued
    Split split;
    Walk walk;    // behind the first piece
    Piece first;
    int2 sums[16];
    float warps[4][64];  // per row, of each softmax warp of its group: a tile's maxima, a piece's sums
    float factor[64];    // what O^T's columns are multiplied with
    float ref[64];
};

// Over the softmax warps.
template <int THREADS>
__device__ __forceinline__ bool any_softmax(bool x) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.aligned.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x)), "n"(THREADS)
        : "memory");
    return r != 0;
}
template <int THREADS>
__device__ __forceinline__ void sync_softmax() {
    __syncwarp();
    asm volatile("barrier.cta.sync.aligned 1, %0;" ::"n"(THREADS) : "memory");
}

template <int N>
__device__ __forceinline__ void load_scores(uint32_t (&x)[N / 2], uint32_t addr) {
    if constexpr (N == 32) tmem_ld_m4(x, addr);
    if constexpr (N == 16) tmem_ld_m2(x, addr);
}

static_assert(sizeof(Shared) <= 2048, "beside the largest configuration's 225 KB");

template <int R, int N, int CL>
__global__ void __launch_bounds__(Cfg<R, N, CL>::THREADS, 1)
    latent_attention_kernel(const LatentAttentionArgs a, const LatentSplit sp,
                            const __grid_constant__ CUtensorMap mq,
                            const __grid_constant__ CUtensorMap mc) {
    using C = Cfg<R, N, CL>;
    constexpr int kThreads = C::THREADS, kSoft = 32 * C::SW;
    extern __shared__ unsigned char raw[];
    __shared__ Shared sh;
    unsigned char *base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    unsigned char *q_smem = base + C::STAGES * C::STAGE;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = a.n_q_heads;
    const int worker = blockIdx.x / CL;
    const int rank = blockIdx.x % CL;
    int4 *records = static_cast<int4 *>(a.workspace);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            for (int x = 0; x < C::PARTS; ++x) {
                mbar_init(&sh.full[s][x], 1);
                mbar_init(&sh.empty[s][x], 1);
            }
        }
        mbar_init(&sh.s_full[0], 1);
        mbar_init(&sh.s_full[1], 1);
        mbar_init(&sh.p_ready[0], C::SW);
        mbar_init(&sh.p_ready[1], C::SW);
        mbar_init(&sh.pv_done[0], 1);
        mbar_init(&sh.pv_done[1], 1);
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.o_full, 1);
        mbar_init(&sh.o_free, C::SW);
        mbar_init(&sh.drained[0], 1);
        mbar_init(&sh.drained[1], 1);
        sh.stop = sh.begun = sh.asked = 0;
        sh.first.tiles = 0;
        fence_barrier_init();
    }
    if (warp == C::SW + 1) {
        tmem_alloc(&sh.tmem, C::TMEM);
        if (lane == 0) {
            prefetch_tmap(&mq);
            prefetch_tmap(&mc);
        }
    }
    {
        // the tables come to L2 while the kernel before drains (a prefetch reads
        // nothing that could be stale)
        const long long line = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
        if (line * 32 < static_cast<long long>(a.num_seqs) * a.max_blocks_per_seq)
            prefetch_l2(a.block_tables + line * 32);
        if (blockIdx.x == 0 && line * 32 <= a.num_seqs) {
            if (line * 32 < a.num_seqs) prefetch_l2(a.context_lens + line * 32);
            if (a.query_start) prefetch_l2(a.query_start + line * 32);
        }
    }
    grid_dependency_wait();
    allow_dependent_launch();

    // the split: every CTA sums the units of all sequences and finds its range
    {
        const int per = (a.num_seqs + kThreads - 1) / kThreads;
        const int b0 = min(static_cast<int>(threadIdx.x) * per, a.num_seqs);
        const int b1 = min(b0 + per, a.num_seqs);
        int2 mine = make_int2(0, 0);  // units, segments
        Seq seq;  // the thread's only sequence, where it has one
        for (int b = b0; b < b1; ++b) {
            if (load_seq(a, b, &seq)) {
                mine.x += seq_units(seq, a.n_q_heads, C::ROWS);
                mine.y += row_tiles(seq.n, a.n_q_heads, C::ROWS);
            } else if (blockIdx.x == 0) {
                flag_error(a.err, PKV_ERRBIT_CONTEXT);
            }
        }
        // inclusive scan: within the warp by shuffles, over the warps in shared memory
        int2 acc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, acc.x, o), y = __shfl_up_sync(0xffffffffu, acc.y, o);
            if (lane >= o) {
                acc.x += x;
                acc.y += y;
            }
        }
        if (lane == 31) sh.sums[warp] = acc;
        __syncthreads();
        int before = acc.x - mine.x, total = 0, seg = acc.y - mine.y, segs = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const int2 v = sh.sums[w];
            if (w < warp) {
                before += v.x;
                seg += v.y;
            }
            total += v.x;
            segs += v.y;
        }
        if (blockIdx.x == 0 && sp.by_segment)  // places that no segment has
            for (int i = segs * CL + threadIdx.x; i < sp.records * CL; i += kThreads)
                records[i] = make_int4(0, 0, 0, 0);
        const int workers = min(total, sp.workers);
        if (worker < workers) {
            const Split split{total / workers, total % workers};
            const int first = split.first(worker);
            if (before <= first && first < before + mine.x) {
                int b = b0, at = before;
                if (per > 1)
                    for (;; ++b) {
                        if (!load_seq(a, b, &seq)) continue;
                        const int u = seq_units(seq, a.n_q_heads, C::ROWS);
                        if (first < at + u) break;
                        at += u;
                        seg += row_tiles(seq.n, a.n_q_heads, C::ROWS);
                    }
                // the first piece, for all roles at once
                Walk w{b, 0, first - at, split.first(worker + 1) - first, at, seg};
                Piece p;
                piece_of(seq, a.n_q_heads, C::ROWS, &w, &p);
                sh.split = split;
                sh.walk = w;
                sh.first = p;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    volatile int *stop = &sh.stop;
    Walk w = sh.walk;
    Piece p = sh.first;

    if (p.tiles == 0) {
        if (threadIdx.x == 0 && !sp.by_segment) records[blockIdx.x] = make_int4(0, 0, 0, 0);
    } else if (warp == C::SW) {
        // --- copies ---
        // a lane looks up `box` tokens of a tile, which one block holds
        constexpr int kMost = kTile / 16;  // boxes of a tile, at most
        const int box = min(a.block_size, kTile), boxes = kTile / box;
        const char *cache = static_cast<const char *>(a.cache);
        const int block_log2 = 31 - __clz(a.block_size);
        // a worker of one CTA reads its tiles once: first to leave L2.  Unshared blocks
        // gain (32 x 128 .. 2048 tokens x 16 heads 20.2 -> 19.0 us, 64 x 1000 .. 3000
        // 37.9 -> 37.4, the same with latents of 256 23.8 -> 21.8), a prefix that many
        // sequences share loses (32 or 64 behind 2048 tokens nothing, 64 behind 8192
        // 85.8 -> 89.5, 200 x 32 heads behind 4096 172 -> 184).  The tiles of a worker of
        // two CTAs stay for the other one.
        const uint64_t policy = l2_policy_evict_first();
        int g = 0, k = 0;  // tiles, pieces so far
        int begun = 0;     // parts of tiles so far
        int asked = 0;     // copies of queries so far
        bool ok = true;
        do {
            const int32_t *table = a.block_tables + static_cast<long long>(p.b) * a.max_blocks_per_seq;
            const int end = p.t0 + p.tiles;
            constexpr int kNone = INT_MIN;
            auto block_of = [&](int t) {  // this lane's entry of the table for tile t
                const int token = t * kTile + lane * box;
                return lane >= boxes || token >= p.s.len || t >= end ? kNone : table[token >> block_log2];
            };
            auto row_of = [&](int t, int id) {  // its first cache row, or -1
                if (id == kNone) return -1;
                if (id < 0 || id >= a.num_blocks) {
                    flag_error(a.err, PKV_ERRBIT_BLOCK_ID);
                    id = 0;  // some block of the pool: the sequence's result is unspecified
                }
                return (id << block_log2) + ((t * kTile + lane * box) & (a.block_size - 1));
            };
            auto to_l2 = [&](int row) {
                const int part = box / CL;  // the worker's CTAs fetch a part of each box
                if (row >= 0)
                    bulk_prefetch_l2(cache + static_cast<long long>(row + rank * part) * (C::E * 2),
                                     part * C::E * 2);
            };
            // entries are looked up an iteration before they are used (a lookup takes as
            // long as half a tile), and at the start all at once, before any is checked
            int ahead[kAhead + 2];  // tiles t .. t + 1 + kAhead
#pragma unroll
            for (int d = 0; d < kAhead + 2; ++d) ahead[d] = block_of(p.t0 + d);
            if (lane == 0) {
                ok = wait_or_stop(&sh.q_empty, (k & 1) ^ 1, stop);
                if (ok) {
                    ++asked;
                    mbar_arrive_expect_tx(&sh.q_full, C::Q_BYTES);
                    const int row = p.s.q0 * H + p.rt * C::ROWS + rank * N;
                    for (int x = 0; x < N / 8; ++x)
                        tma_load_3d(q_smem + x * C::Q_GROUP, &mq, 0, row + 8 * x, 0, &sh.q_full);
                }
            }
            ++k;
            for (int t = p.t0; t < end; ++t, ++g) {
                const int s = g % C::STAGES, row = row_of(t, ahead[0]);
                const int live = __popc(__ballot_sync(0xffffffffu, row >= 0));
                // one lane issues: a copy issued by several lanes costs some 100 cycles a lane
                int groups[kMost];  // of 8 cache rows, or -1
#pragma unroll
                for (int i = 0; i < kMost; ++i) {
                    const int r = __shfl_sync(0xffffffffu, row, i);
                    groups[i] = r >= 0 ? r / 8 : -1;
                }
                if (elect_one()) {
                    unsigned char *dst = base + s * C::STAGE;
#pragma unroll 1
                    for (int x = 0; x < C::PARTS; ++x) {
                        ok = poll_or_stop(&sh.empty[s][x], ((g / C::STAGES) & 1) ^ 1, stop);
                        if (!ok) break;
                        // only now: a part's bytes announced while its place still had
                        // copies of the tile before in flight would count for those
                        uint64_t *full = &sh.full[s][x];
                        if (live > 0)
                            mbar_arrive_expect_tx(full, live * (box / 8) * C::GROUP);
                        else
                            mbar_arrive(full);
#pragma unroll
                        for (int i = 0; i < kMost; ++i) {
                            if (groups[i] < 0) continue;
                            unsigned char *to = dst + x * C::PART + i * (box / 8) * C::GROUP;
                            if (CL > 1)
                                tma_load_4d(to, &mc, 0, 0, x * C::PP, groups[i], full);
                            else
                                tma_load_4d(to, &mc, 0, 0, x * C::PP, groups[i], full, policy);
                        }
                        begun = C::PARTS * g + x + 1;
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (t == p.t0)
#pragma unroll
                    for (int d = 1; d < kAhead; ++d) to_l2(row_of(t + d, ahead[d]));
                to_l2(row_of(t + kAhead, ahead[kAhead]));
#pragma unroll
                for (int d = 0; d < kAhead + 1; ++d) ahead[d] = ahead[d + 1];
                ahead[kAhead + 1] = block_of(t + 2 + kAhead);
            }
            ok = __all_sync(0xffffffffu, ok);
        } while (ok && next_piece(a, C::ROWS, &w, &p));
        begun = __reduce_max_sync(0xffffffffu, begun);
        if (lane == 0) {
            sh.begun = begun;
            sh.asked = asked;
        }
    } else if (warp == C::SW + 1) {
        // --- scores ---
        // One warp issues them, the next one the outputs' products: neither's waits
        // and commits keep the tensor core from the other's work.
        if (elect_one()) {
            constexpr uint32_t ds = mma_desc(kTile, N, false, false);
            const uint32_t kv = smem_addr(base);
            const uint64_t qd = smem_desc(smem_addr(q_smem), C::Q_GROUP, 0);
            int g = 0, k = 0;
            bool ok = first_wait(&sh.full[0][0], 0, a.first_wait_polls, stop);
            do {
                ok = ok && wait_or_stop(&sh.q_full, k & 1, stop);
#pragma unroll 1
                for (int j = 0; j < p.tiles && ok; ++j, ++g) {
                    // the scores' place is free when the weights before last are made
                    if (g > 1) ok = wait_or_stop(&sh.p_ready[g & 1], ((g >> 1) & 1) ^ 1, stop);
                    if (!ok) break;
                    const uint64_t kd = smem_desc(kv + (g % C::STAGES) * C::STAGE, C::GROUP, 0);
                    const uint32_t d = tmem + (C::VT + (g & 1)) * N;
#pragma unroll
                    for (int part = 0; part < C::PARTS; ++part) {
                        ok = ok && poll_or_stop(&sh.full[g % C::STAGES][part], (g / C::STAGES) & 1, stop);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int x = 4 * C::PP * part; x < 4 * C::PP * (part + 1); ++x)
                            mma_ss(d, kd + C::plane(x / 4) / 16 + (x % 4) * 2, qd + (x / 4) * 64 + (x % 4) * 2,
                                   ds, x > 0);
                    }
                    if (!ok) break;
                    mma_commit(&sh.s_full[g & 1]);
                }
                if (ok) mma_commit(&sh.q_empty);
                ++k;
            } while (ok && next_piece(a, C::ROWS, &w, &p));
            // nothing of the tensor core is left in flight when TMEM is freed
            mma_commit(&sh.drained[0]);
            mbar_wait_bounded(&sh.drained[0], 0);
        }
    } else if (warp == C::SW + 2) {
        // --- outputs' products ---
        if (elect_one()) {
            constexpr uint32_t dpv = mma_desc(128, N, true, true);
            const uint32_t kv = smem_addr(base);
            int g = 0, k = 0;
            bool ok = true;
            do {
                ok = wait_or_stop(&sh.o_free, (k & 1) ^ 1, stop);
#pragma unroll 1
                for (int j = 0; j < p.tiles && ok; ++j, ++g) {
                    ok = poll_or_stop(&sh.p_ready[g & 1], (g >> 1) & 1, stop);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t va = kv + (g % C::STAGES) * C::STAGE;
                    const uint64_t pd = smem_desc(va + C::P_AT, C::GROUP, 0);
#pragma unroll
                    for (int v = 0; v < C::VT; ++v) {
                        const uint64_t vd = smem_desc(va + C::plane(2 * v), C::GROUP,
                                                      C::plane(2 * v + 1) - C::plane(2 * v));
#pragma unroll
                        for (int x = 0; x < kTile / 16; ++x)
                            mma_ss(tmem + v * N, vd + 2 * x * C::GROUP / 16,
                                   pd + 2 * x * C::GROUP / 16, dpv, j > 0 || x > 0);
#pragma unroll
                        for (int part = 0; part < C::PARTS; ++part) {
                            if (C::last_reader(part) != v) continue;
                            mma_commit(&sh.empty[g % C::STAGES][part]);
                        }
                    }
                    mma_commit(&sh.pv_done[g & 1]);
                }
                if (ok) mma_commit(&sh.o_full);
                ++k;
            } while (ok && next_piece(a, C::ROWS, &w, &p));
            mma_commit(&sh.drained[1]);
            mbar_wait_bounded(&sh.drained[1], 0);
        }
    } else {
        // --- softmax, results ---
        // scores: this thread holds tokens tok (+ 8) and rows row_of(c) (+ 1), c < NC
        constexpr int NC = C::NG / 8;
        const int group = warp >> 2, quarter = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(quarter) << 21;
        const int tok = 16 * quarter + lane / 4, col = C::NG * group + 2 * (lane & 3);
        const Layout lay = layout(sp.records, sp.workers, CL, N, R);
        char *ws = static_cast<char *>(a.workspace);
        const float scale = a.scale_log2, unscale = 1.f / scale;
        int g = 0, k = 0;
        bool recorded = false;
        do {
            const int tile_row = p.rt * C::ROWS + rank * N;  // of the sequence's rows
            float ref[NC][2], sum[NC][2], most[NC][2];  // most: scores above it move ref
            int seen[NC][2];  // tokens that the row attends
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    seen[c][e] = p.s.len;
                    if (p.s.n > 1)
                        seen[c][e] = min(p.s.len - p.s.n + (tile_row + 8 * c + col + e) / H + 1, p.s.len);
                    ref[c][e] = sum[c][e] = most[c][e] = 0.f;
                }
            // tiles below this one need no mask
            const int first_masked =
                (p.s.n == 1 ? p.s.len : p.s.len - p.s.n + min(tile_row / H + 1, p.s.n)) / kTile;
            for (int j = 0; j < p.tiles; ++j, ++g) {
                const int t = p.t0 + j;
                warp_wait_or_stop(&sh.s_full[g & 1], (g >> 1) & 1, stop);
                tc_fence_after();
                uint32_t xr[C::NG / 2];
                load_scores<C::NG>(xr, tmem + (C::VT + (g & 1)) * N + C::NG * group + lanes);
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
                        top[c][e] = fmaxf(x[c][e], x[c][2 + e]);
                        move |= top[c][e] > most[c][e];
                    }
                if (any_softmax<kSoft>(move)) {
                    // new references: the tile's maxima over all tokens
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1)
                                top[c][e] = fmaxf(top[c][e], __shfl_xor_sync(0xffffffffu, top[c][e], o));
                            if (lane < 4) sh.warps[quarter][8 * c + col + e] = top[c][e];
                        }
                    sync_softmax<kSoft>();
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int n = 8 * c + col + e;
                            const float m = fmaxf(fmaxf(sh.warps[0][n], sh.warps[1][n]),
                                                  fmaxf(sh.warps[2][n], sh.warps[3][n])) * scale;
                            float next = ref[c][e];
                            if (j == 0)
                                next = m > -INFINITY ? m - kHead : 0.f;
                            else if (m - next > kHead + kLag)
                                next = m - kHead;
                            const float f = j == 0 ? 1.f : ex2(ref[c][e] - next);
                            sum[c][e] *= f;
                            ref[c][e] = next;
                            most[c][e] = (next + kHead + kLag) * unscale;
                            if (quarter == 0 && lane < 4) sh.factor[n] = f;
                        }
                    sync_softmax<kSoft>();
                    if (j > 0) {
                        // O^T's columns follow, after the products into it
                        warp_wait_or_stop(&sh.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, stop);
                        tc_fence_after();
#pragma unroll 1
                        for (int v = 16 * group; v < C::VT * N; v += 16 * C::GROUPS) {
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
                    const float2 u = fma2(make_float2(x[c][0], x[c][2]), scale, -ref[c][0]);
                    const float2 v = fma2(make_float2(x[c][1], x[c][3]), scale, -ref[c][1]);
                    const float p0 = ex2(u.x), p1 = ex2(v.x), p2 = ex2(u.y), p3 = ex2(v.y);
                    sum[c][0] += p0 + p2;
                    sum[c][1] += p1 + p3;
                    y[c][0] = pack_half2(p0, p1);
                    y[c][1] = pack_half2(p2, p3);
                }
                unsigned char *tile = base + (g % C::STAGES) * C::STAGE;
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = tok + 8 * e, piece = c + NC * group;
                        *reinterpret_cast<uint32_t *>(tile + (r / 8) * C::GROUP + C::P_AT +
                                                      (r % 8) * 128 + ((piece ^ (r & 7)) << 4) +
                                                      4 * (lane & 3)) = y[c][e];
                    }
                // values of rows past the sequence's end meet weights of 0: they must
                // be finite
                const int valid = p.s.len - t * kTile;
                if (valid < kTile) {
                    for (int e = threadIdx.x; e < (kTile - valid) * (R / 8); e += kSoft) {
                        const int r = valid + e / (R / 8), piece = e % (R / 8);
                        *reinterpret_cast<uint4 *>(tile + C::plane(piece / 8) + (r / 8) * C::GROUP +
                                                   (r % 8) * 128 + (piece % 8) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    // The products of two tiles before are done when these weights are
                    // announced: a wait names its phase by parity alone, so no barrier
                    // may get two phases ahead of who waits for it, or the softmax two
                    // tiles ahead of the products.  A ring of two tiles has no room for
                    // that (there the wait would cost 64 x 128 heads 1.7 %).
                    if (C::STAGES > 2 && g > 1)
                        wait_or_stop(&sh.pv_done[g & 1], ((g >> 1) & 1) ^ 1, stop);
                    mbar_arrive(&sh.p_ready[g & 1]);
                }
            }
            // the row sums, over the tokens of all threads
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1)
                        sum[c][e] += __shfl_xor_sync(0xffffffffu, sum[c][e], o);
                    if (lane < 4) sh.warps[quarter][8 * c + col + e] = sum[c][e];
                    if (quarter == 0 && lane < 4) sh.ref[8 * c + col + e] = ref[c][e];
                }
            warp_wait_or_stop(&sh.o_full, k & 1, stop);
            tc_fence_after();
            sync_softmax<kSoft>();
            const int rows = min(N, p.s.n * H - tile_row);  // this CTA's; none: padding
            const int row0 = p.s.q0 * H + tile_row;
            const bool whole = p.t0 == 0 && p.tiles == p.seg_tiles;
            const int slot = (2 * worker + (p.t0 == 0 ? 1 : 0)) * CL + rank;
            if (static_cast<int>(threadIdx.x) < rows) {
                const int n = threadIdx.x;
                const float l = (sh.warps[0][n] + sh.warps[1][n]) + (sh.warps[2][n] + sh.warps[3][n]);
                if (whole) {
                    sh.factor[n] = l == 0.f ? 0.f : 1.f / l;
                    if (a.lse_out)
                        a.lse_out[row0 + n] =
                            l == 0.f ? -INFINITY : (sh.ref[n] + log2f(l)) * 0.69314718055994531f;
                } else {
                    reinterpret_cast<float2 *>(ws + lay.ml)[static_cast<size_t>(slot) * N + n] =
                        make_float2(l == 0.f ? -INFINITY : sh.ref[n], l);
                }
            }
            if (whole) {
                sync_softmax<kSoft>();
                __half *out = static_cast<__half *>(a.out) + static_cast<long long>(row0) * R +
                              32 * quarter + lane;
#pragma unroll 1
                for (int v = 16 * group; v < C::VT * N; v += 16 * C::GROUPS) {
                    const int n0 = v % N;
                    if (n0 >= rows) continue;
                    uint32_t o[16];
                    tmem_ld16(o, tmem + v + lanes);
                    tmem_wait_ld();
                    __half *dst = out + n0 * R + 128 * (v / N);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (n0 + e < rows)
                            dst[e * R] = __float2half_rn(__uint_as_float(o[e]) * sh.factor[n0 + e]);
                }
            } else {
                uint4 *acc = reinterpret_cast<uint4 *>(ws + lay.acc) +
                             static_cast<size_t>(slot) * (N / 4 * R) + 32 * quarter + lane;
#pragma unroll 2
                for (int v = 16 * group; v < C::VT * N; v += 16 * C::GROUPS) {
                    uint32_t o[16];
                    tmem_ld16(o, tmem + v + lanes);
                    tmem_wait_ld();
                    uint4 *dst = acc + (v % N) / 4 * R + 128 * (v / N);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dst[e * R] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
            }
            tc_fence_before();
            sync_softmax<kSoft>();  // sh.warps, sh.ref and sh.factor are free again
            if (lane == 0) mbar_arrive(&sh.o_free);
            if (p.t0 == 0) {
                // the worker that starts a segment says where its last piece is
                if (threadIdx.x == 0 && (!whole || sp.by_segment)) {
                    const int at = sp.by_segment ? p.seg : worker;
                    const int last = whole ? worker : sh.split.worker_of(p.seg_first + p.seg_tiles - 1);
                    records[at * CL + rank] = make_int4(row0, whole ? 0 : max(rows, 0), worker, last);
                }
                recorded |= !whole;
            }
            ++k;
        } while (next_piece(a, C::ROWS, &w, &p));
        if (!recorded && threadIdx.x == 0 && !sp.by_segment) records[blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && sh.stop) {
        flag_error(a.err, PKV_ERRBIT_TIMEOUT);
        // Every copy in flight lands before the CTA gives its memory back.  Not until here:
        // the copy role may have issued its last one before another role gave up.
        if (sh.asked > 0) mbar_wait_bounded(&sh.q_full, (sh.asked - 1) & 1);
        for (int i = max(0, sh.begun - C::PARTS * C::STAGES); i < sh.begun; ++i) {
            const int t = i / C::PARTS;
            mbar_wait_bounded(&sh.full[t % C::STAGES][i % C::PARTS], (t / C::STAGES) & 1);
        }
    }
    __syncwarp();
    if (warp == C::SW + 1) tmem_free(tmem, C::TMEM);
}

// The pieces of each cut segment, joined.  A unit is four rows of one column (one
// 16-byte load a piece).  A block has 256 / G * U neighbouring columns of four rows,
// U a thread, and G threads for each of them, which take every G-th piece.
constexpr int kJoinThreads = 256;

template <int R, int N, int CL, int U>
__global__ void __launch_bounds__(kJoinThreads, 4)
    latent_join_kernel(const LatentAttentionArgs a, const LatentSplit sp) {
    __shared__ float parts[kJoinThreads / 32][4], warp_l[kJoinThreads / 32][4];
    __shared__ float row_ref[4], row_inv[4];
    __shared__ float4 sums[U][kJoinThreads];
    grid_dependency_wait();
    allow_dependent_launch();
    const int4 rec = static_cast<const int4 *>(a.workspace)[blockIdx.x];
    const int G = sp.join_threads, units = kJoinThreads / G;
    const int at0 = static_cast<int>(blockIdx.y) * units * U;  // the block's first unit
    const int n0 = at0 / R * 4;  // the block's rows
    if (n0 >= rec.y) return;
    const Layout lay = layout(sp.records, sp.workers, CL, N, R);
    const char *ws = static_cast<const char *>(a.workspace);
    const float2 *ml = reinterpret_cast<const float2 *>(ws + lay.ml) + n0;
    const float4 *acc = reinterpret_cast<const float4 *>(ws + lay.acc);
    const int pieces = rec.w - rec.z + 1, rank = blockIdx.x % CL;
    auto slot = [&](int k) { return static_cast<size_t>((2 * (rec.z + k) + (k == 0 ? 1 : 0)) * CL + rank); };
    // this block's first loads of partial sums need nothing of the rows' statistics
    const int u = threadIdx.x % units, i = threadIdx.x / units;
    float4 first[U];
#pragma unroll
    for (int c = 0; c < U; ++c)
        first[c] = i < pieces ? acc[slot(i) * (N / 4 * R) + at0 + c * units + u]
                              : make_float4(0.f, 0.f, 0.f, 0.f);
    // the rows' references and sums over all pieces: thread x takes row x % 4 of every
    // 64th piece
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float m = -INFINITY, l = 0.f;
    for (int k = threadIdx.x / 4; k < pieces; k += kJoinThreads / 4) {
        const float2 v = ml[slot(k) * N + threadIdx.x % 4];
        const float next = fmaxf(m, v.x);
        if (next > -INFINITY) l = l * ex2(m - next) + v.y * ex2(v.x - next);
        m = next;
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
        const float next = fmaxf(m, m2);
        if (next > -INFINITY) l = l * ex2(m - next) + l2 * ex2(m2 - next);
        m = next;
    }
    if (lane < 4) {
        parts[warp][lane] = m;
        warp_l[warp][lane] = l;
    }
    __syncthreads();
    if (threadIdx.x < 4) {
        float r = -INFINITY, t = 0.f;
#pragma unroll
        for (int x = 0; x < kJoinThreads / 32; ++x) r = fmaxf(r, parts[x][threadIdx.x]);
        r = r > -INFINITY ? r : 0.f;
#pragma unroll
        for (int x = 0; x < kJoinThreads / 32; ++x)
            t += warp_l[x][threadIdx.x] * ex2(parts[x][threadIdx.x] - r);
        row_ref[threadIdx.x] = r;
        row_inv[threadIdx.x] = t == 0.f ? 0.f : 1.f / t;
        const int n = n0 + threadIdx.x;
        if (a.lse_out && at0 % R == 0 && n < rec.y)
            a.lse_out[rec.x + n] = t == 0.f ? -INFINITY : (r + log2f(t)) * 0.69314718055994531f;
    }
    __syncthreads();
    float ref[4], inv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        ref[e] = row_ref[e];
        inv[e] = row_inv[e];
    }
    float4 s[U];
#pragma unroll
    for (int c = 0; c < U; ++c) s[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll(U > 1 ? 1 : 4)
    for (int k = i; k < pieces; k += G) {
        const size_t sl = slot(k);
        float4 v[U];
#pragma unroll
        for (int c = 0; c < U; ++c) v[c] = k == i ? first[c] : acc[sl * (N / 4 * R) + at0 + c * units + u];
        const float4 ma = *reinterpret_cast<const float4 *>(ml + sl * N);
        const float4 mb = *reinterpret_cast<const float4 *>(ml + sl * N + 2);
        const float f0 = ex2(ma.x - ref[0]), f1 = ex2(ma.z - ref[1]);
        const float f2 = ex2(mb.x - ref[2]), f3 = ex2(mb.z - ref[3]);
#pragma unroll
        for (int c = 0; c < U; ++c) {
            s[c].x = fmaf(v[c].x, f0, s[c].x);
            s[c].y = fmaf(v[c].y, f1, s[c].y);
            s[c].z = fmaf(v[c].z, f2, s[c].z);
            s[c].w = fmaf(v[c].w, f3, s[c].w);
        }
    }
    if (G > 1) {
#pragma unroll
        for (int c = 0; c < U; ++c) sums[c][threadIdx.x] = s[c];
        __syncthreads();
        if (i > 0) return;
#pragma unroll
        for (int c = 0; c < U; ++c)
            for (int k = 1; k < G; ++k) {
                const float4 v = sums[c][k * units + u];
                s[c].x += v.x;
                s[c].y += v.y;
                s[c].z += v.z;
                s[c].w += v.w;
            }
    }
    __half *out = static_cast<__half *>(a.out) + (static_cast<long long>(rec.x) + n0) * R + at0 % R + u;
#pragma unroll
    for (int c = 0; c < U; ++c) {
        const float y[4] = {s[c].x * inv[0], s[c].y * inv[1], s[c].z * inv[2], s[c].w * inv[3]};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n0 + e < rec.y) out[e * R + c * units] = __float2half_rn(y[e]);
    }
}

// Rows of `width` fp16 values, as 64 columns x 8 rows x planes (x groups of 8 rows,
// where the rows are a multiple of 8 and copied from such a row on): a box is 8 rows of
// `planes` planes, plane by plane, `groups` times over, with the 128-byte swizzle.
bool make_map(CUtensorMap *m, const void *base, cuuint64_t rows, cuuint64_t width, cuuint32_t planes,
              cuuint32_t groups) {
    auto fn = encode_fn();
    const cuuint64_t dims[4] = {64, groups ? 8 : rows, width / 64, rows / 8};
    const cuuint64_t strides[3] = {width * 2, 128, width * 16};
    const cuuint32_t box[4] = {64, 8, planes, groups}, one[4] = {1, 1, 1, 1};
    return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, groups ? 4 : 3, const_cast<void *>(base), dims,
                    strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int R, int N, int CL>
cudaError_t launch(const LatentAttentionArgs &a, const LatentSplit &sp, cudaStream_t stream) {
    using C = Cfg<R, N, CL>;
    CUtensorMap mq, mc;
    if (!make_map(&mq, a.q, static_cast<cuuint64_t>(a.total_q) * a.n_q_heads, C::E, C::PL, 0) ||
        !make_map(&mc, a.cache, static_cast<cuuint64_t>(a.num_blocks) * a.block_size, C::E, C::PP,
                  (a.block_size < kTile ? a.block_size : kTile) / 8))
        return cudaErrorNotSupported;
    auto kern = latent_attention_kernel<R, N, CL>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t attr = allow_smem(kern, C::SMEM, done);
    if (attr != cudaSuccess) return attr;
    const cudaError_t e = launch_pdl(kern, dim3(sp.workers * CL), dim3(C::THREADS), C::SMEM, stream, a,
                                     sp, mq, mc);
    if (e != cudaSuccess) return e;
    // more columns a thread where the rows are many: fewer, longer blocks
    constexpr int U = N == 64 ? R / 256 : 1;
    const dim3 grid(sp.records * CL, R * N / 4 * sp.join_threads / (kJoinThreads * U));
    return launch_pdl(latent_join_kernel<R, N, CL, U>, grid, dim3(kJoinThreads), 0, stream, a, sp);
}

}  // namespace

bool latent_split(int num_seqs, int max_q_len, int heads, int latent_dim, int max_len, int sms,
                  LatentSplit *sp) {
    const long long rows = static_cast<long long>(max_q_len) * heads;
    sp->rows = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    sp->ctas = rows > 64 ? 2 : 1;
    const int tile = sp->rows * sp->ctas;
    const long long tiles = (rows + tile - 1) / tile;
    const long long units = tiles * num_seqs * (max_len / kTile + 1);
    if (units >= (1LL << 31)) return false;
    sp->workers = sms / sp->ctas;
    // few segments: a record each; more than workers: one for what each worker starts
    sp->by_segment = tiles * num_seqs <= sp->workers;
    sp->records = sp->by_segment ? static_cast<int>(tiles * num_seqs) : sp->workers;
    // threads of the join over a segment's pieces, about workers / segments of them: a
    // quarter to a half of the pieces; with 64 rows half of that, as its blocks are many
    // anyway (measured: 16 x 4 tokens x 32 heads 44.3 us with 2 threads, 42.6 with 1; 32
    // sequences x 16 heads 20.5 with 2, 21.0 with 1)
    const long long segments = tiles * num_seqs > 0 ? tiles * num_seqs : 1;
    const long long pieces = sp->workers / segments / (sp->rows == 64 ? 2 : 1);
    sp->join_threads = pieces >= 16 ? 8 : pieces >= 8 ? 4 : pieces >= 4 ? 2 : 1;
    sp->ws_bytes = layout(sp->records, sp->workers, sp->ctas, sp->rows, latent_dim).total;
    return true;
}

cudaError_t launch_latent_attention(const LatentAttentionArgs &a, const LatentSplit &sp,
                                    cudaStream_t stream) {
    if (a.latent_dim == 512)
        return sp.ctas == 2 ? launch<512, 64, 2>(a, sp, stream)
               : sp.rows == 16 ? launch<512, 16, 1>(a, sp, stream)
               : sp.rows == 32 ? launch<512, 32, 1>(a, sp, stream)
                               : launch<512, 64, 1>(a, sp, stream);
    return sp.ctas == 2 ? launch<256, 64, 2>(a, sp, stream)
           : sp.rows == 16 ? launch<256, 16, 1>(a, sp, stream)
           : sp.rows == 32 ? launch<256, 32, 1>(a, sp, stream)
                           : launch<256, 64, 1>(a, sp, stream);
}

}  // namespace pkv
