// q8_attention.cu -- attention over the 8-bit caches with block scales for up to 32 query
// rows of a KV head: decode, few drafts (paged_decode_attention_q8).
//
// Mathematics.  For the query rows of one KV head (tokens x heads of its group) and a
// tile of 16 cached tokens of one block, with codes K, V and the block's scales k, v:
//
//   S^T = K Q^T               16 tokens x rows, codes widened to fp16 (exact), fp32 sums
//   s   = S * (k * scale * log2 e)
//   p   = 2^(s - m)           m: the row's reference
//   l  += p,   O^T += V^T (p * (v / w))^T        w: the warp's V reference
//
// and the result is O w / l.  Tokens are the M side of the first product and value
// columns that of the second, so up to 8 rows fill an 8-wide N and no tensor-core row
// is empty.  m moves only when a logit is 2^8 above it, w when v leaves [w / 64, 16 w]:
// both are vote-and-branch, and p * (v / w) stays within fp16.
//
// Layout.  Each warp has a ring of tiles of its own, filled by TMA, one copy a tile of K
// and one of V, swizzled.  The order of entries inside a product is free (K's columns go
// with Q's, V's columns are rows of the result), so a lane's 16 contiguous bytes of a row
// are its operand, every read is conflict-free, and the result leaves in 16 contiguous
// entries a lane.  V's token pairs are interleaved by one byte permute per four codes
// before they are widened.  (16-byte cp.async into places of the lane's own, without
// swizzle or barrier, was bound by the cycle that each 32-byte sector takes on its way
// into shared memory: 8 x 32k tokens 110 us.)
//
// Split.  The (sequence, head, 16-token tile) units are cut into equal ranges for the
// warps of one CTA per SM.  The parts of a segment (sequence, head) that several warps of
// a CTA hold are joined there; CTAs that share a segment leave a record each, and the
// last to arrive joins them, in the order of the tokens.
//
// Measured (32 query heads on 8 of 128, E4M3): 8 x 32k tokens 87 us, 6.2 TB/s, memory; 32 x
// 128 to 2048 tokens 21.0 us, 3.4 TB/s, of which 4 us pass before the first tile lands and 5 us in the
// joins; 20 rows, 24 x 200 to 2900 tokens, 36.2 us, where a warp's chain of instructions bounds
// it (255 registers a thread, two warps a scheduler).
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "q8.h"
#include "q8_codes.cuh"
#include "rope_latent.h"

namespace pkv {
namespace {

constexpr int kTile = 16;   // tokens of a unit
constexpr float kMoveM = 8.f;            // a row's reference follows logits this far above it
constexpr float kLn2 = 0.69314718055994531f;
// Units a warp gets at least, where there are enough: a shorter range spends its time
// in the join.
constexpr int kMinUnits = 2;

// Floats of a record: sums and two numbers a row, whole 16-byte pieces.
__host__ __device__ constexpr int q8_record_floats(int rows, int d) { return rows * d + (rows + 1) / 2 * 4; }

template <int D, int NT>
struct Shape {
    // Registers bound the warps: the sums take NT * D / 4 of a lane's.  At NT = 1 (32 x
    // 128-2048 tokens; 8 x 32k; one of 700): 8 warps, 5 stages 21.6, 102, 8.1 us; 12 and 3:
    // 21.0, 87.4, 9.2; 16 and 2: 20.9, 87.4, 10.9.
    static constexpr int kWarps = NT <= 2 ? 12 : 8;
    static constexpr int kStages = NT == 1 || NT == 3 ? 3 : 2;
    static constexpr int kRows = 8 * NT;
    static constexpr bool kQInRegs = NT == 1;           // one tile of rows; else read from shared memory for each tile
    static constexpr int kVPiece = D / 8;               // bytes of a V row a lane takes
    static constexpr int kV = kTile * D;                // of V in a stage
    static constexpr int kStage = 2 * kTile * D;
    // A warp's shared memory: the ring, then two places for Q: a segment's that is ahead,
    // and one more ahead or the one in use, if that is not in registers.  A warp's last
    // record takes it all over.
    static constexpr int kQ = kStages * kStage, kQBytes = NT * D * 16;
    static constexpr int kQAhead = kQInRegs ? 2 : 1;
    static constexpr int kWarpBytes = kQ + 2 * kQBytes;
    static_assert(q8_record_floats(kRows, D) * 4 <= kWarpBytes, "the last record's place");
    static_assert(kWarpBytes % 1024 == 0, "swizzled tiles lie on 1024 bytes");
    static constexpr size_t smem(int seqs) { return kWarps * kWarpBytes + (static_cast<size_t>(seqs) * 3 + 2) * 4; }
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All groups have landed but the `newer` (0 to 2) last ones.
__device__ __forceinline__ void wait_copies(int newer) {
    if (newer == 0)
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (newer == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 2;" ::: "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// x / d for x < 2^31: the high part of a product (Divide's comment has the bound).
__device__ __forceinline__ int divided(int x, const Q8Divide &d) {
    return static_cast<int>(static_cast<unsigned long long>(static_cast<unsigned>(x)) * d.mul >> d.shift);
}

// `total` units in `n` ranges whose sizes differ by one at most, the larger first.
struct Ranges {
    int size, larger;  // of a smaller range; how many larger ones
    __device__ Ranges(int total, int n) : size(total / n), larger(total - size * n) {}
    __device__ int start(int i) const { return size * i + min(i, larger); }
    __device__ int of(int x) const {  // the range that unit x lies in
        const int split = larger * (size + 1);
        return x < split ? x / (size + 1) : larger + (x - split) / max(size, 1);
    }
};

// A batch's units: sequence b has those from cum[b] to cum[b + 1].
struct Batch {
    const int *cum, *len, *start;  // shared memory
    int total;
};

// One segment, with the warp's place in it.
struct Segment {
    int b, h;   // sequence, KV head
    int tiles;  // of the sequence
    int j;      // 16-token tile

    // The unit u of the batch.
    __device__ void find(const Batch &t, const Q8AttentionArgs &a, int u) {
        int lo = 0, hi = a.num_seqs;  // cum[lo] <= u < cum[hi]
#pragma unroll 1
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (t.cum[mid] <= u) lo = mid; else hi = mid;
        }
        b = lo;
        tiles = (t.len[b] + kTile - 1) / kTile;
        j = u - t.cum[b];
        h = j / tiles;
        j -= h * tiles;
    }
    // The next unit; true when it is another segment's first.
    __device__ bool next(const Batch &t, const Q8AttentionArgs &a) {
        if (++j < tiles) return false;
        j = 0;
        if (++h < a.n_kv_heads) return true;
        h = 0;
#pragma unroll 1
        do ++b; while (b < a.num_seqs && t.cum[b + 1] == t.cum[b]);
        if (b < a.num_seqs) tiles = (t.len[b] + kTile - 1) / kTile;
        return true;
    }
    // The unit at which the segment starts, given that u is its unit j.
    __device__ int first(int u) const { return u - j; }
};

// The cache tile (number of 16-row pieces) of unit u; bad blocks flag and become tile 0.
__device__ __forceinline__ unsigned tile_of(const Batch &t, const Q8AttentionArgs &a, int bs16_log2, int u,
                                            Segment &s) {
    s.find(t, a, u);
    const int block = s.j >> bs16_log2;
    const int id = a.block_tables[static_cast<long long>(s.b) * a.max_blocks_per_seq + block];
    if (id < 0 || id >= a.num_blocks) {
        flag_error(a.err, PKV_ERRBIT_BLOCK_ID);
        return 0;
    }
    return (static_cast<unsigned>(id) * a.n_kv_heads + s.h << bs16_log2) + (s.j & ((1 << bs16_log2) - 1));
}

// Where query row `row` of a segment lies, as a multiple of head_dim in out; -1: its rows end
// before it.
__device__ __forceinline__ long long row_at(const Batch &t, const Q8AttentionArgs &a, int b, int h, int group,
                                            int row, int *token) {
    const int i = divided(row, a.by_group);
    *token = i;
    if (i >= t.start[b + 1] - t.start[b]) return -1;
    return static_cast<long long>(t.start[b] + i) * a.n_q_heads + h * group + (row - i * group);
}

// A row of a segment joined by 8 lanes: lane i of them holds the columns 32 k + 4 i on.
template <int D>
struct Row {
    float4 sum[D / 32];
    float top = -INFINITY, weight = 0.f;

    __device__ Row() {
#pragma unroll
        for (int k = 0; k < D / 32; ++k) sum[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // Another reference, at least the one there is.
    __device__ void move(float to) {
        const float g = top == -INFINITY ? 0.f : ex2(top - to);  // 0 of nothing
        top = to;
        weight *= g;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            sum[k].x *= g;
            sum[k].y *= g;
            sum[k].z *= g;
            sum[k].w *= g;
        }
    }
    __device__ void add(float m, float l, const float4 (&x)[D / 32]) {
        const float g = m == -INFINITY ? 0.f : ex2(m - top);
        weight += g * l;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            sum[k].x += g * x[k].x;
            sum[k].y += g * x[k].y;
            sum[k].z += g * x[k].z;
            sum[k].w += g * x[k].w;
        }
    }
    __device__ void write(const Q8AttentionArgs &a, long long row, int i) const {
        const float z = 1.f / weight;
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
            reinterpret_cast<uint2 *>(a.out)[row * (D / 4) + k * 8 + i] =
                make_uint2(pack_half2(sum[k].x * z, sum[k].y * z), pack_half2(sum[k].z * z, sum[k].w * z));
        if (a.lse_out && i == 0) a.lse_out[row] = (top + log2f(weight)) * kLn2;
    }
};

// From shared memory or from L2, whatever the address says; never from L1.
__device__ __forceinline__ float4 load_fresh4(const float *p) {
    float4 x;
    asm volatile("ld.volatile.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(p) : "memory");
    return x;
}
__device__ __forceinline__ float2 load_fresh2(const float *p) {
    float2 x;
    asm volatile("ld.volatile.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "l"(p) : "memory");
    return x;
}

// What a warp leaves of a segment that it holds a part of.
struct Piece {
    int first, end;  // the segment's units; first -1: none
    int b, h;
    int in_ring;     // the record is in the warp's shared memory, else in the workspace
};

template <int KIND, int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kWarps * 32, 1) q8_attention_kernel(
    const Q8AttentionArgs a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using S = Shape<D, NT>;
    constexpr int kRows = S::kRows, kWarps = S::kWarps;
    extern __shared__ __align__(1024) unsigned char smem[];
    int *cum = reinterpret_cast<int *>(smem + kWarps * S::kWarpBytes);
    int *len = cum + a.num_seqs + 1, *start = len + a.num_seqs;
    __shared__ int warp_sums[kWarps];
    __shared__ Piece pieces[kWarps * 2];
    __shared__ uint64_t landed[kWarps][S::kStages];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int r = lane / 4, c = lane % 4;  // the lane's row and column in a fragment
    const int group = a.n_q_heads / a.n_kv_heads;
    const int bs16_log2 = __ffs(a.block_size / kTile) - 1;

    if (threadIdx.x == 0) {
        prefetch_tmap(&k_map);
        prefetch_tmap(&v_map);
    }
    if (lane < S::kStages) mbar_init(&landed[warp][lane], 1);
    fence_barrier_init();
    // the block tables into L2, a line a thread of the grid (a prefetch reads nothing stale)
    const long long line = static_cast<long long>(blockIdx.x) + static_cast<long long>(threadIdx.x) * gridDim.x;
    if (line * 32 < static_cast<long long>(a.num_seqs) * a.max_blocks_per_seq) prefetch_l2(a.block_tables + line * 32);
    if (!a.tables_ready) {
        grid_dependency_wait();
        allow_dependent_launch();
    }

    // --- the batch's units
    int total = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.num_seqs; b0 += kWarps * 32) {
        const int b = b0 + threadIdx.x;
        int units = 0;
        if (b < a.num_seqs) {
            int n = 1, l = a.context_lens[b], s = b;
            if (a.query_start) {
                s = a.query_start[b];
                n = a.query_start[b + 1] - s;
            } else if (l == 0) {
                n = 0;
            }
            const bool ok = n >= 0 && n <= a.max_q_len && n <= l && s >= 0 && s <= a.total_q - n &&
                            l <= a.max_context_len;
            if (!ok && blockIdx.x == 0) flag_error(a.err, PKV_ERRBIT_CONTEXT);
            if (ok) units = n > 0 ? (l + kTile - 1) / kTile * a.n_kv_heads : 0;
            len[b] = l;
            start[b] = s;
            if (b == a.num_seqs - 1) start[b + 1] = s + n;
        }
        int upto = units;  // sum over the warp, this thread included
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int z = __shfl_up_sync(~0u, upto, d);
            if (lane >= d) upto += z;
        }
        if (b0 > 0) __syncthreads();  // the sums of the round before are read
        if (lane == 31) warp_sums[warp] = upto;
        __syncthreads();
        int before = total;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int x = warp_sums[w];
            if (w < warp) before += x;
            total += x;
        }
        if (b < a.num_seqs) cum[b] = before + upto - units;
    }
    if (threadIdx.x == 0) cum[a.num_seqs] = total;
    if (lane < 2) pieces[2 * warp + lane].first = -1;
    __syncthreads();
    const Batch t{cum, len, start, total};

    // --- this warp's range
    const int ctas = min(static_cast<int>(gridDim.x), max(1, (total + kWarps * kMinUnits - 1) / (kWarps * kMinUnits)));
    const int cta = blockIdx.x;
    const Ranges of_ctas(total, ctas);
    const int U0 = cta < ctas ? of_ctas.start(cta) : 0, U1 = cta < ctas ? of_ctas.start(cta + 1) : 0;
    const Ranges of_warps(U1 - U0, kWarps);
    const int u0 = U0 + of_warps.start(warp), u1 = U0 + of_warps.start(warp + 1);

    // --- what copies need: 32 units' tiles at a time, the next 32 under way
    int base = u0;
    unsigned tiles_now = 0, tiles_next = 0;
    Segment seg{};  // of unit u0: lane 0's, for all
    if (u0 + lane < u1) tiles_now = tile_of(t, a, bs16_log2, u0 + lane, seg);
    seg.b = __shfl_sync(~0u, seg.b, 0);
    seg.h = __shfl_sync(~0u, seg.h, 0);
    seg.j = __shfl_sync(~0u, seg.j, 0);
    seg.tiles = __shfl_sync(~0u, seg.tiles, 0);
    if (a.tables_ready) {
        grid_dependency_wait();
        allow_dependent_launch();
    }

    unsigned char *mine = smem + warp * S::kWarpBytes;
    uint64_t *full = landed[warp];
    Segment ahead = seg;
    int pu = u0;         // the next unit to copy
    int pstage = 0, pq = 0, pending = 0;
    bool pfirst = true;  // it starts a segment, or this range
    bool alive = true;   // no wait has given up
    float2 scales_prev = make_float2(0.f, 0.f), scales_now = scales_prev;
    auto load_scales = [&] {
        scales_prev = scales_now;
        if (base + lane < u1) {
            const unsigned cell = tiles_now >> bs16_log2;
            scales_now = make_float2(__ldcg(a.k_scales + cell), __ldcg(a.v_scales + cell));
        }
    };

    auto copy_tile = [&](bool does, unsigned tile, int to_stage) {
        if (does) {
            unsigned char *dst = mine + to_stage * S::kStage;
            mbar_arrive_expect_tx(full + to_stage, S::kStage);
            tma_load_2d(dst, &k_map, 0, static_cast<int>(tile * kTile), full + to_stage);
            tma_load_2d(dst + S::kV, &v_map, 0, static_cast<int>(tile * kTile), full + to_stage);
        }
    };
    // Copies of the units before `to`, as far as there are places for their queries; the
    // first tile is under way.
    auto copy_ahead = [&](int to) {
#pragma unroll 1
        while (pu < to && !(pfirst && pending == S::kQAhead) && alive) {
            if (pu - base == 32) {
                base += 32;
                tiles_now = tiles_next;
                load_scales();
            }
            const unsigned tile = __shfl_sync(~0u, tiles_now, pu - base);
            if (pu > u0) copy_tile(lane == 0, tile, pstage);
            if (pu == base && base + 32 + lane < u1) {
                Segment any;
                tiles_next = tile_of(t, a, bs16_log2, base + 32 + lane, any);
            }
            if (pfirst) {
                const uint32_t dst = smem_addr(mine) + S::kQ + pq * S::kQBytes + lane * 16;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    int token;
                    const long long row = row_at(t, a, ahead.b, ahead.h, group, nt * 8 + r, &token);
                    const int head = ahead.h * group + (nt * 8 + r - token * group);
                    const __half *q = static_cast<const __half *>(a.q) +
                                      (row < 0 ? 0 : (t.start[ahead.b] + token) * a.q_stride + head * D) + c * (D / 4);
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        copy16(dst + (nt * (D / 32) + i) * 512, q + i * 8, row < 0 ? 0 : 16);
                }
                commit();
                pq ^= 1;
                ++pending;
            }
            ++pu;
            pfirst = ahead.next(t, a);
            pstage = pstage + 1 == S::kStages ? 0 : pstage + 1;
        }
    };

    // the first tile; its queries come before the next ones, or they would wait behind them
    copy_tile(lane == 0 && u0 < u1, tiles_now, 0);
    load_scales();
    if (!a.query_start) {  // one token a sequence: an empty one has a result
#pragma unroll 1
        for (int b = blockIdx.x; b < a.num_seqs; b += gridDim.x) {
            if (len[b] != 0) continue;
            uint4 *o = static_cast<uint4 *>(a.out) + static_cast<long long>(b) * a.n_q_heads * (D / 8);
#pragma unroll 1
            for (int i = threadIdx.x; i < a.n_q_heads * (D / 8); i += kWarps * 32) o[i] = make_uint4(0, 0, 0, 0);
            if (a.lse_out)
#pragma unroll 1
                for (int i = threadIdx.x; i < a.n_q_heads; i += kWarps * 32)
                    a.lse_out[static_cast<long long>(b) * a.n_q_heads + i] = -INFINITY;
        }
    }
    // Records, `record_rows` sums of D, then m and l of each row: of the CTA's warps that went
    // on after it, then of the segment that began in a CTA before, and of the one that goes
    // on in the next.
    unsigned char *ws = static_cast<unsigned char *>(a.workspace);
    auto record_of = [&](int of_cta, int i) {
        return reinterpret_cast<float *>(ws + kBalancedCounterBytes) +
               ((kWarps + 2ll) * of_cta + i) * q8_record_floats(a.record_rows, D);
    };

    // the lane's places in a tile: K rows r (and r + 8, 8 rows on), V rows 2c and 2c + 1 (and
    // 8 rows on), by the TMA swizzle of D-byte rows
    const int k0 = D == 128 ? r * D + (2 * c ^ r) * 16 : r * D + (c ^ (r >> 1)) * 16;
    const int k1 = r * D + (2 * c + 1 ^ r) * 16;
    const int v0 = S::kV + 2 * c * D + (D == 128 ? (r ^ 2 * c) * 16 : ((r >> 1) ^ c) * 16 + (r & 1) * 8);
    const int v1 = S::kV + (2 * c + 1) * D + (D == 128 ? (r ^ 2 * c + 1) * 16 : ((r >> 1) ^ c) * 16 + (r & 1) * 8);
    int stage = 0, parity = 0, qplace = 0;
    int polls = a.first_wait_polls;  // test hook: from 0 on, polls of the first wait before it gives up
#pragma unroll 1
    for (int u = u0; u < u1;) {
        // --- a piece of a segment: units u to end
        const int seg_first = seg.first(u), seg_end = seg_first + seg.tiles, end = min(seg_end, u1);
        const int L = len[seg.b], n = start[seg.b + 1] - start[seg.b];
        uint32_t q[1][D / 16][2];
        float o[NT][D / 16][4], l[NT][2], m[NT][2];
        int limit[NT][2];  // keys that a row attends
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][mt][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[nt][i] = 0.f;
                m[nt][i] = -INFINITY;
                limit[nt][i] = L - n + 1 + min(divided(nt * 8 + 2 * c + i, a.by_group), n - 1);
            }
        }
        const int least = L - n + 1;  // of the first row
        float w = 0.f, inv_w = 0.f;
        const unsigned char *qp = mine + S::kQ + qplace * S::kQBytes + lane * 16;
        qplace ^= 1;
        bool first = true;
#pragma unroll 1
        for (; u < end; ++u) {
            copy_ahead(min(u + S::kStages, u1));  // into the stage read last time
            if (first) {
                first = false;
                --pending;
                wait_copies(pending);
                if constexpr (S::kQInRegs) {
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(qp + i * 512);
                        q[0][2 * i][0] = x.x;
                        q[0][2 * i][1] = x.y;
                        q[0][2 * i + 1][0] = x.z;
                        q[0][2 * i + 1][1] = x.w;
                    }
                }
            }
            if (alive) {
                const bool ok = polls >= 0 ? polls > 0 && mbar_wait_polls(full + stage, parity, polls - 1)
                                           : mbar_wait_bounded(full + stage, parity);
                polls = -1;
                if (!__all_sync(~0u, ok)) {
                    // results are unspecified from here on, but every step of the split is made
                    if (lane == 0) flag_error(a.err, PKV_ERRBIT_TIMEOUT);
                    alive = false;
                    const int sent = max(pu, min(u0 + 1, u1));
#pragma unroll 1
                    for (int k = u, s = stage, y = parity; k < sent; ++k) {  // no copy outlives the warp
                        mbar_wait_bounded(full + s, y);
                        if (++s == S::kStages) s = 0, y ^= 1;
                    }
                    __syncwarp();
                }
            }
            const unsigned char *p = mine + stage * S::kStage;
            if (++stage == S::kStages) stage = 0, parity ^= 1;
            const int tok = (u - seg_first) * kTile;
            const bool past = u < base;
            const float k_scale = __shfl_sync(~0u, past ? scales_prev.x : scales_now.x, (u - base) & 31);
            const float v_scale = __shfl_sync(~0u, past ? scales_prev.y : scales_now.y, (u - base) & 31);
            const float f = k_scale * a.scale_log2;
            // --- scores, in two sums (half as long a chain)
            float s[NT][4], s2[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[nt][i] = s2[nt][i] = 0.f;
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {
                const uint4 x = *reinterpret_cast<const uint4 *>(p + (half ? k1 : k0));
                const uint4 y = *reinterpret_cast<const uint4 *>(p + (half ? k1 : k0) + 8 * D);
                const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int ii = 0; ii < 2; ++ii) {
                    uint4 qx[NT];
                    if constexpr (!S::kQInRegs) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            qx[nt] = *reinterpret_cast<const uint4 *>(qp + (nt * (D / 32) + 2 * half + ii) * 512);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int i = 2 * ii + k;
                        const uint32_t frag[4] = {q8_widen<KIND, 0>(wx[i]), q8_widen<KIND, 0>(wy[i]),
                                                  q8_widen<KIND, 1>(wx[i]), q8_widen<KIND, 1>(wy[i])};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            uint32_t b0, b1;
                            if constexpr (S::kQInRegs) {
                                b0 = q[nt][half * 4 + i][0];
                                b1 = q[nt][half * 4 + i][1];
                            } else {
                                b0 = k ? qx[nt].z : qx[nt].x;
                                b1 = k ? qx[nt].w : qx[nt].y;
                            }
                            mma_16816(k ? s2[nt] : s[nt], frag, b0, b1);
                        }
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[nt][i] = (s[nt][i] + s2[nt][i]) * f;
            if (tok + kTile > least) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (tok + r + (i >> 1) * 8 >= limit[nt][i & 1]) s[nt][i] = -INFINITY;
            }
            // --- references
            bool move = v_scale > 0.f && !(v_scale >= w * (1.f / 64.f) && v_scale <= w * 16.f);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) move = move || s[nt][i] > m[nt][i & 1] + kMoveM;
            if (__any_sync(~0u, move)) {
                float g = 1.f;
                if (v_scale > 0.f && !(v_scale >= w * (1.f / 64.f) && v_scale <= w * 16.f)) {
                    const float to = fmaxf(v_scale, kQ8LeastReference);
                    inv_w = __fdividef(1.f, to);
                    g = w * inv_w;
                    w = to;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float h[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float top = fmaxf(s[nt][i], s[nt][i + 2]);
#pragma unroll
                        for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                        const float to = fmaxf(m[nt][i], top);
                        h[i] = m[nt][i] == -INFINITY ? 0.f : ex2(m[nt][i] - to);
                        m[nt][i] = to;
                        l[nt][i] *= h[i];
                        h[i] *= g;
                    }
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[nt][mt][i] *= h[i & 1];
                }
            }
            // --- weights
            const float fv = v_scale * inv_w;
            uint32_t pf[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // a row that has attended nothing yet has no reference
                    const float ref = m[nt][i & 1] == -INFINITY ? 0.f : m[nt][i & 1];
                    e[i] = ex2(s[nt][i] - ref);
                    l[nt][i & 1] += e[i];
                }
                pf[nt][0] = transposed(pack_half2(e[0] * fv, e[1] * fv));
                pf[nt][1] = transposed(pack_half2(e[2] * fv, e[3] * fv));
            }
            // --- outputs: tokens 2c, 2c + 1 (x) and 2c + 8, 2c + 9 (y) of the lane's columns
            uint32_t v[4][S::kVPiece / 4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const unsigned char *src = p + (i & 1 ? v1 : v0) + (i >> 1) * 8 * D;
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(src);
                    v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(src);
                    v[i][0] = x.x; v[i][1] = x.y;
                }
            }
            if (tok + kTile > L) {  // rows that hold no token may hold anything
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (tok + 2 * c + (i & 1) + (i >> 1) * 8 >= L)
#pragma unroll
                        for (int k = 0; k < S::kVPiece / 4; ++k) v[i][k] = 0;
            }
#pragma unroll
            for (int k = 0; k < S::kVPiece / 4; ++k)
#pragma unroll
                for (int hi = 0; hi < 2; ++hi) {
                    const uint32_t sel = hi ? 0x7362 : 0x5140;
                    const uint32_t x = __byte_perm(v[0][k], v[1][k], sel), y = __byte_perm(v[2][k], v[3][k], sel);
                    const uint32_t frag[4] = {q8_widen<KIND, 0>(x), q8_widen<KIND, 1>(x), q8_widen<KIND, 0>(y),
                                              q8_widen<KIND, 1>(y)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_16816(o[nt][2 * k + hi], frag, pf[nt][0], pf[nt][1]);
                }
            __syncwarp();  // every lane has read this stage
        }
        // --- the piece's end: sums over the lanes of a row
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int d = 4; d < 32; d *= 2) l[nt][i] += __shfl_xor_sync(~0u, l[nt][i], d);
        if (seg_first >= u0 && seg_end <= u1) {  // whole
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    int token;
                    const long long row = row_at(t, a, seg.b, seg.h, group, nt * 8 + 2 * c + i, &token);
                    if (row < 0) continue;
                    const float z = w / l[nt][i];
                    __half *dst = static_cast<__half *>(a.out) + row * D + r * S::kVPiece;
                    uint32_t y[D / 16];
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt) y[mt] = pack_half2(o[nt][mt][i] * z, o[nt][mt][i + 2] * z);
#pragma unroll
                    for (int k = 0; k < D / 64; ++k)
                        reinterpret_cast<uint4 *>(dst)[k] =
                            make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
                    if (a.lse_out && r == 0) a.lse_out[row] = (m[nt][i] + log2f(l[nt][i])) * kLn2;
                }
        } else {
            // --- a part.  The last thing that the warp does takes its shared memory (no copy
            // is in flight any more); what it goes on after goes to the workspace
            const int valid = n * group;
            __syncwarp();
            float *rec = end == u1 ? reinterpret_cast<float *>(mine) : record_of(cta, warp);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = nt * 8 + 2 * c + i;
                    if (row >= valid) continue;
#pragma unroll
                    for (int k = 0; k < D / 32; ++k)
                        *reinterpret_cast<float4 *>(rec + row * D + r * S::kVPiece + 4 * k) =
                            make_float4(o[nt][2 * k][i] * w, o[nt][2 * k][i + 2] * w, o[nt][2 * k + 1][i] * w,
                                        o[nt][2 * k + 1][i + 2] * w);
                    if (r == 0)
                        *reinterpret_cast<float2 *>(rec + a.record_rows * D + 2 * row) = make_float2(m[nt][i], l[nt][i]);
                }
            if (lane == 0)
                pieces[2 * warp + (seg_first >= u0)] = Piece{seg_first, seg_end, seg.b, seg.h, end == u1};
        }
        if (u < u1) {
            seg.j = seg.tiles - 1;
            seg.next(t, a);
        }
    }
    __syncthreads();

    // --- joins.  Lane i knows piece i; pieces of one segment are neighbours, in the order of
    // the tokens.  A warp takes four rows of a segment, 8 lanes each.
    static_assert(2 * kWarps <= 32, "a lane for each piece");
    const int my_first = lane < 2 * kWarps ? pieces[lane].first : -1;
    const unsigned there = __ballot_sync(~0u, my_first >= 0);
    const unsigned lower = there & ((1u << lane) - 1);
    const int prev = __shfl_sync(~0u, my_first, lower ? 31 - __clz(lower) : 0);
    const unsigned heads = __ballot_sync(~0u, my_first >= 0 && (!lower || prev != my_first));
    const int segments = __popc(heads);
    constexpr int kQuads = kRows / 4;
#pragma unroll 1
    for (int item = warp; item < segments * kQuads; item += kWarps) {
        unsigned of = heads;
        int quad = 0, nth = item;
        while (nth >= segments) nth -= segments, quad += 4;
        for (; nth > 0; --nth) of &= of - 1;
        const int head = __ffs(of) - 1;
        const unsigned rest = of & (of - 1);
        unsigned members = there & (rest ? (rest & -rest) - 1 : ~0u) & ~((1u << head) - 1);
        const Piece at = pieces[head];
        const int valid = (start[at.b + 1] - start[at.b]) * group;
        if (quad >= valid) continue;
        const int row = min(quad + lane / 8, valid - 1), i8 = lane % 8;
        const int side = at.first >= U0;
        bool whole = side && at.end <= U1;
        int from = 0, parts = 0;  // of the CTAs', on the second round
#pragma unroll 1
        while (true) {
            Row<D> y;
            constexpr int kAtOnce = 4;  // loads go out for so many parts together
#pragma unroll 1
            for (int k0 = 0; parts ? k0 < parts : members != 0; k0 += kAtOnce) {
                float4 x[kAtOnce][D / 32];
                float2 ml[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const float *rec;
                    bool there_is;
                    if (parts) {
                        there_is = k0 + k < parts;
                        rec = record_of(from + k0 + k, kWarps + (k0 + k == 0));
                    } else {
                        there_is = members != 0;
                        const int p = there_is ? __ffs(members) - 1 : head;
                        members &= members - 1;
                        rec = pieces[p].in_ring ? reinterpret_cast<const float *>(smem + p / 2 * S::kWarpBytes)
                                                : static_cast<const float *>(record_of(cta, p / 2));
                    }
                    ml[k] = make_float2(-INFINITY, 0.f);
                    if (there_is) {
#pragma unroll
                        for (int j = 0; j < D / 32; ++j) x[k][j] = load_fresh4(rec + row * D + j * 32 + i8 * 4);
                        ml[k] = load_fresh2(rec + a.record_rows * D + 2 * row);
                    } else {
#pragma unroll
                        for (int j = 0; j < D / 32; ++j) x[k][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                }
                float top = y.top;
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, ml[k].x);
                y.move(top);
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) y.add(ml[k].x, ml[k].y, x[k]);
            }
            if (whole) {
                int token;
                const long long out_row = row_at(t, a, at.b, at.h, group, row, &token);
                if (quad + lane / 8 < valid) y.write(a, out_row, i8);
                break;
            }
            // other CTAs share the segment: the last to arrive with these rows joins them
            float *part = record_of(cta, kWarps + side);
            if (quad + lane / 8 < valid) {
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                    __stcg(reinterpret_cast<float4 *>(part + row * D) + j * 8 + i8, y.sum[j]);
                if (i8 == 0)
                    __stcg(reinterpret_cast<float2 *>(part + a.record_rows * D) + row, make_float2(y.top, y.weight));
            }
            __syncwarp();
            from = of_ctas.of(at.first);
            parts = of_ctas.of(at.end - 1) - from + 1;
            if (lane == 0) {
                int *counter = reinterpret_cast<int *>(ws) + from * kQuads + quad / 4;
                const int old = atomic_add_acq_rel_gpu(counter, 1);
                if (counter_not_zeroed(old, parts - 1)) {
                    flag_error(a.err, PKV_ERRBIT_WORKSPACE);
                    atomic_exch_relaxed_gpu(counter, kCounterPoison);
                } else if (old == parts - 1) {
                    whole = true;
                    red_add_relaxed_gpu(counter, -parts);
                }
            }
            whole = __shfl_sync(~0u, whole, 0);
            __syncwarp();  // lane 0's acquire before every lane's loads of the other CTAs' records
            if (!whole) break;
        }
    }
}

template <int KIND, int D, int NT>
cudaError_t launch(const Q8AttentionArgs &a, const Q8Split &sp, cudaStream_t stream) {
    const size_t smem = Shape<D, NT>::smem(a.num_seqs);
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(q8_attention_kernel<KIND, D, NT>,
                                     static_cast<int>(Shape<D, NT>::smem(kQ8MaxSeqs)), done);
    if (e != cudaSuccess) return e;
    CUtensorMap k_map, v_map;
    const long long rows = a.num_blocks * a.n_kv_heads * a.block_size;
    if (!make_cache_map_e4m3(&k_map, a.k_cache, rows, D) || !make_cache_map_e4m3(&v_map, a.v_cache, rows, D))
        return cudaErrorNotSupported;
    return launch_pdl(q8_attention_kernel<KIND, D, NT>, dim3(sp.ctas), dim3(Shape<D, NT>::kWarps * 32), smem,
                      stream, a, k_map, v_map);
}

template <int KIND, int D>
cudaError_t launch_rows(const Q8AttentionArgs &a, const Q8Split &sp, cudaStream_t stream) {
    switch (sp.row_tiles) {
        case 1: return launch<KIND, D, 1>(a, sp, stream);
        case 2: return launch<KIND, D, 2>(a, sp, stream);
        case 3: return launch<KIND, D, 3>(a, sp, stream);
        default: return launch<KIND, D, 4>(a, sp, stream);
    }
}

template <int NT>
constexpr bool fits() {
    return Shape<128, NT>::smem(kQ8MaxSeqs) <= 227 * 1024 - 1024;
}
static_assert(fits<1>() && fits<2>() && fits<3>() && fits<4>(), "shared memory");

}  // namespace

namespace {

constexpr int kFewRows = 32;

// The split of up to that many rows of a KV head.
Q8Split split_of_rows(int rows, int head_dim, int sms) {
    Q8Split sp{};
    sp.row_tiles = (rows + 7) / 8;
    const int warps = sp.row_tiles <= 2 ? Shape<128, 2>::kWarps : Shape<128, 4>::kWarps;
    static_assert(Shape<128, 1>::kWarps == Shape<128, 2>::kWarps && Shape<128, 3>::kWarps == Shape<128, 4>::kWarps, "");
    const int most = kBalancedMaxWorkers / (2 * sp.row_tiles);  // a counter for four rows of each
    sp.ctas = std::min(sms, most);
    sp.record_rows = rows;
    sp.ws_bytes = kBalancedCounterBytes +
                  static_cast<size_t>(sp.ctas) * (warps + 2) * q8_record_floats(rows, head_dim) * sizeof(float);
    return sp;
}

// Up to 32 rows here, more on tcgen05.  This kernel and that one, us, 8 KV heads, at 12, 20 and 32 rows:
//   24 x 200-2900 tokens   E4M3, 128  25.9 49.3, 36.0 48.6, 46.5 47.7   int8, 64  21.1 42.2, 30.5 41.4, 36.1 41.1
//   2 x 30000              E4M3, 128  35.7 68.7, 47.8 69.0, 57.3 64.4   int8, 64  29.4 55.6, 39.4 55.9, 43.6 52.8
//   8 x 32000              E4M3, 128   102 178,   145 178,   178 177    int8, 64  85.7 157,   119 158,   134 157
// (int8 of 128: 188 and 210 for the last, E4M3 of 64: 131 and 154.)  64 rows of the first, twice 32
// here: 55.1, 49.3
long long rows_of(int max_q_len, int n_q_heads, int n_kv_heads) {
    return static_cast<long long>(max_q_len) * (n_q_heads / n_kv_heads);
}

}  // namespace

bool q8_fits(int num_seqs, int max_q_len, int n_q_heads, int n_kv_heads, int max_len) {
    if (rows_of(max_q_len, n_q_heads, n_kv_heads) > kFewRows)
        return q8_prefill_fits(num_seqs, max_q_len, n_q_heads, n_kv_heads, max_len);
    return static_cast<double>(num_seqs) * n_kv_heads * ((static_cast<double>(max_len) + kTile - 1) / kTile) <= kQ8MaxUnits;
}

Q8Split q8_split(int max_q_len, int n_q_heads, int n_kv_heads, int head_dim, int sms) {
    const long long rows = rows_of(max_q_len, n_q_heads, n_kv_heads);
    return rows > kFewRows ? q8_prefill_split(max_q_len, n_q_heads, n_kv_heads, head_dim, sms)
                           : split_of_rows(static_cast<int>(rows), head_dim, sms);
}

size_t q8_plan_bytes(int max_q_len, int n_q_heads, int n_kv_heads, int head_dim, int sms) {
    const long long rows = rows_of(max_q_len, n_q_heads, n_kv_heads);
    // fewer rows may take more: they have more warps, whose records are apart
    size_t bytes = rows > kFewRows ? q8_prefill_split(max_q_len, n_q_heads, n_kv_heads, head_dim, sms).ws_bytes : 0;
    for (int r = 1; r <= kFewRows && r <= rows; ++r) bytes = std::max(bytes, split_of_rows(r, head_dim, sms).ws_bytes);
    return bytes;
}

cudaError_t launch_q8_attention(const Q8AttentionArgs &a, int kind, const Q8Split &sp,
                                cudaStream_t stream) {
    if (sp.row_tiles == 0) return launch_q8_prefill(a, kind, sp, stream);
    if (a.head_dim == 128)
        return kind == PKV_Q8_E4M3 ? launch_rows<PKV_Q8_E4M3, 128>(a, sp, stream)
                                   : launch_rows<PKV_Q8_INT8, 128>(a, sp, stream);
    return kind == PKV_Q8_E4M3 ? launch_rows<PKV_Q8_E4M3, 64>(a, sp, stream)
                               : launch_rows<PKV_Q8_INT8, 64>(a, sp, stream);
}

}  // namespace pkv
