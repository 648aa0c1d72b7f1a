// q8_attention.cu -- attention over the 8-bit caches with block scales
// (paged_decode_attention_q8).
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
// Layout.  A lane copies what it will use itself, and nothing else, with 16-byte
// cp.async into its own places of a ring: no barrier and no exchange between lanes,
// and conflict-free reads.  The order of entries inside a product is free (K's columns
// go with Q's, V's columns are rows of the result), so a lane's 16 contiguous bytes of a
// row are its operand, and the result leaves in 16 contiguous entries a lane.  V's token
// pairs are interleaved by one byte permute per four codes before they are widened.
//
// Split.  The (sequence, head, row tile, 16-token tile) units are cut into equal ranges
// for the warps of one CTA per SM.  Pieces of a segment (sequence, head, row tile) that
// several warps hold join in shared memory; those of several CTAs leave one record a
// CTA, and the last CTA to arrive joins the records in order.
#include <cuda_fp16.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "q8.h"
#include "q8_codes.cuh"

namespace pkv {
namespace {

constexpr int kTile = 16;   // tokens of a unit
constexpr int kWarps = 8;
constexpr float kMoveM = 8.f;            // a row's reference follows logits this far above it
constexpr float kLn2 = 0.69314718055994531f;
// Units a warp gets at least, where there are enough: a shorter range spends its time
// in the join.
constexpr int kMinUnits = 2;

template <int D, int NT>
struct Shape {
    static constexpr int kRows = 8 * NT;
    static constexpr int kKPieces = D / 32;             // 16-byte pieces of K a lane (2 rows)
    static constexpr int kVPiece = D / 8;               // bytes of a V row a lane takes
    static constexpr int kQPieces = NT * D / 32;        // 16-byte pieces of Q a lane
    static constexpr int kV = kKPieces * 512;           // offsets in a stage
    static constexpr int kQ = kV + 4 * kVPiece * 32;
    static constexpr int kS = kQ + kQPieces * 512;
    static constexpr int kStage = kS + 256;
    static constexpr int kStages = NT == 1 ? 3 : 2;
    static constexpr int kRecord = kRows * D + 2 * kRows;  // floats: sums, then m and l a row
    static constexpr int kRingBytes = kWarps * kStages * kStage;
    static constexpr int kRecordBytes = kWarps * kRecord * 4;
    static_assert(kRecord * 4 <= kStages * kStage, "a warp's ring holds its last piece's record");
    static constexpr size_t smem(int seqs) {
        return kRingBytes + kRecordBytes + (static_cast<size_t>(seqs) * 3 + 2) * 4 + kWarps * 64;
    }
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// A batch's units: sequence b has those from cum[b] to cum[b + 1].
struct Batch {
    const int *cum, *len, *start;  // shared memory
    int total;
};

// One segment, with the warp's place in it.
struct Segment {
    int b, h, rt;          // sequence, KV head, row tile
    int tiles, row_tiles;  // of the sequence
    int j;                 // 16-token tile

    // The unit u of the batch.
    __device__ void find(const Batch &t, const Q8AttentionArgs &a, int rows, int group, int u) {
        int lo = 0, hi = a.num_seqs;  // cum[lo] <= u < cum[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (t.cum[mid] <= u) lo = mid; else hi = mid;
        }
        b = lo;
        sizes(t, rows, group);
        int r = u - t.cum[b];
        const int q = r / tiles;
        j = r - q * tiles;
        h = q / row_tiles;
        rt = q - h * row_tiles;
    }
    __device__ void sizes(const Batch &t, int rows, int group) {
        tiles = (t.len[b] + kTile - 1) / kTile;
        row_tiles = ((t.start[b + 1] - t.start[b]) * group + rows - 1) / rows;
    }
    // The next unit; true when it is another segment's first.
    __device__ bool next(const Batch &t, const Q8AttentionArgs &a, int rows, int group) {
        if (++j < tiles) return false;
        j = 0;
        if (++rt < row_tiles) return true;
        rt = 0;
        if (++h < a.n_kv_heads) return true;
        h = 0;
        do ++b; while (b < a.num_seqs && t.cum[b + 1] == t.cum[b]);
        if (b < a.num_seqs) sizes(t, rows, group);
        return true;
    }
    // The unit at which the segment starts, given that u is its unit j.
    __device__ int first(int u) const { return u - j; }
};

// The cache tile (number of 16-row pieces) of unit u; bad blocks flag and become tile 0.
__device__ __forceinline__ unsigned tile_of(const Batch &t, const Q8AttentionArgs &a, int rows, int group,
                                            int bs16_log2, int u) {
    Segment s;
    s.find(t, a, rows, group, u);
    const int block = s.j >> bs16_log2;
    const int id = a.block_tables[static_cast<long long>(s.b) * a.max_blocks_per_seq + block];
    if (id < 0 || id >= a.num_blocks) {
        flag_error(a.err, PKV_ERRBIT_BLOCK_ID);
        return 0;
    }
    return (static_cast<unsigned>(id) * a.n_kv_heads + s.h << bs16_log2) + (s.j & ((1 << bs16_log2) - 1));
}

// Sum over the CTA's warps of x (one value a thread), exclusive; *sum gets the whole.
__device__ __forceinline__ int exclusive_sum(int x, int *warp_sums, int *sum) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int y = x;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int z = __shfl_up_sync(~0u, y, d);
        if (lane >= d) y += z;
    }
    if (lane == 31) warp_sums[warp] = y;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    __syncthreads();
    *sum = all;
    return before + y - x;
}

// Where query row `row` of a segment's row tile lies, as a multiple of head_dim in out;
// -1: the tile's rows end before it.
__device__ __forceinline__ long long row_at(const Batch &t, const Q8AttentionArgs &a, const Segment &s,
                                            int rows, int group, int row, int *token) {
    const int r = s.rt * rows + row, i = r / group;
    *token = i;
    if (i >= t.start[s.b + 1] - t.start[s.b]) return -1;
    return static_cast<long long>(t.start[s.b] + i) * a.n_q_heads + s.h * group + (r - i * group);
}

// What a warp or a CTA leaves of a segment it holds a part of.
struct Piece {
    int first, end;  // the segment's units
    int slot;        // -1: none; 0: the warp's record; 1: its ring
    Segment at;
};

template <int KIND, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, 1) q8_attention_kernel(const Q8AttentionArgs a) {
    using S = Shape<D, NT>;
    constexpr int kRows = S::kRows;
    extern __shared__ __align__(128) unsigned char smem[];
    float *records = reinterpret_cast<float *>(smem + S::kRingBytes);
    int *cum = reinterpret_cast<int *>(smem + S::kRingBytes + S::kRecordBytes);
    int *len = cum + a.num_seqs + 1, *start = len + a.num_seqs;
    __shared__ int warp_sums[kWarps];
    __shared__ Piece pieces[kWarps * 2];
    __shared__ int last_of[2];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int r = lane / 4, c = lane % 4;  // the lane's row and column in a fragment
    const int group = a.n_q_heads / a.n_kv_heads;
    const int bs16_log2 = __ffs(a.block_size / kTile) - 1;

    if (!a.tables_ready) {
        grid_dependency_wait();
        allow_dependent_launch();
    }

    // --- the batch's units
    int at = 0;
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
            const bool ok = n >= 0 && n <= a.max_q_len && n <= l && s >= 0 && s + n <= a.total_q &&
                            l <= a.max_context_len;
            if (!ok && blockIdx.x == 0) flag_error(a.err, PKV_ERRBIT_CONTEXT);
            if (ok) units = (l + kTile - 1) / kTile * ((n * group + kRows - 1) / kRows) * a.n_kv_heads;
            len[b] = l;
            start[b] = s;
            if (b == a.num_seqs - 1) start[b + 1] = s + n;
        }
        int sum;
        const int mine = exclusive_sum(units, warp_sums, &sum);
        if (b < a.num_seqs) cum[b] = at + mine;
        at += sum;
    }
    if (threadIdx.x == 0) cum[a.num_seqs] = at;
    __syncthreads();
    const Batch t{cum, len, start, at};
    const int total = at;

    // --- this warp's range
    const int ctas = min(static_cast<int>(gridDim.x), max(1, (total + kWarps * kMinUnits - 1) / (kWarps * kMinUnits)));
    const int cta = blockIdx.x;
    const bool works = cta < ctas;
    auto cut = [&](int i) { return static_cast<int>(static_cast<long long>(total) * i / ctas); };
    const int U0 = works ? cut(cta) : 0, U1 = works ? cut(cta + 1) : 0;
    const int u0 = U0 + static_cast<int>(static_cast<long long>(U1 - U0) * warp / kWarps);
    const int u1 = U0 + static_cast<int>(static_cast<long long>(U1 - U0) * (warp + 1) / kWarps);

    // --- what copies need: 32 units' tiles at a time, the next 32 under way
    int base = u0;
    unsigned tiles_now = 0, tiles_next = 0;
    if (u0 + lane < u1) tiles_now = tile_of(t, a, kRows, group, bs16_log2, u0 + lane);
    if (u0 + 32 + lane < u1) tiles_next = tile_of(t, a, kRows, group, bs16_log2, u0 + 32 + lane);
    if (a.tables_ready) {
        grid_dependency_wait();
        allow_dependent_launch();
    }
    if (!a.query_start) {  // one token a sequence: an empty one has a result
        for (int b = cta; b < a.num_seqs; b += gridDim.x) {
            if (len[b] != 0) continue;
            uint4 *o = static_cast<uint4 *>(a.out) + static_cast<long long>(b) * a.n_q_heads * (D / 8);
            for (int i = threadIdx.x; i < a.n_q_heads * (D / 8); i += kWarps * 32) o[i] = make_uint4(0, 0, 0, 0);
            if (a.lse_out)
                for (int i = threadIdx.x; i < a.n_q_heads; i += kWarps * 32)
                    a.lse_out[static_cast<long long>(b) * a.n_q_heads + i] = -INFINITY;
        }
    }

    const uint32_t ring = smem_addr(smem) + warp * S::kStages * S::kStage;
    unsigned char *ring_p = smem + warp * S::kStages * S::kStage;
    const unsigned char *kc = static_cast<const unsigned char *>(a.k_cache) + r * D + c * 16;
    const unsigned char *vc = static_cast<const unsigned char *>(a.v_cache) + 2 * c * D + r * S::kVPiece;
    Segment ahead;
    int pu = u0;       // the next unit to copy
    int pstage = 0;
    bool pfirst = true;  // it starts a segment, or this range
    if (u0 < u1) ahead.find(t, a, kRows, group, u0);

    auto copy_next = [&] {
        if (pu < u1) {
            if (pu - base == 32) {
                base += 32;
                tiles_now = tiles_next;
                if (base + 32 + lane < u1) tiles_next = tile_of(t, a, kRows, group, bs16_log2, base + 32 + lane);
            }
            const unsigned tile = __shfl_sync(~0u, tiles_now, pu - base);
            const uint32_t dst = ring + pstage * S::kStage;
            const long long off = static_cast<long long>(tile) * (kTile * D);
#pragma unroll
            for (int i = 0; i < S::kKPieces; ++i) {
                // rows r and r + 8; at D = 128 their two halves
                const int row = i & 1, half = i >> 1;
                copy16(dst + i * 512 + lane * 16, kc + off + row * 8 * D + half * 64);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // tokens 2c, 2c + 1, 2c + 8, 2c + 9
                const unsigned char *src = vc + off + ((i & 1) + (i >> 1) * 8) * D;
                if constexpr (D == 128)
                    copy16(dst + S::kV + i * 512 + lane * 16, src);
                else
                    copy8(dst + S::kV + i * 256 + lane * 8, src);
            }
            const unsigned cell = tile >> bs16_log2;
            copy4(dst + S::kS + lane * 8, a.k_scales + cell);
            copy4(dst + S::kS + lane * 8 + 4, a.v_scales + cell);
            if (pfirst) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    int token;
                    const long long row = row_at(t, a, ahead, kRows, group, nt * 8 + r, &token);
                    const int head = static_cast<int>(row % a.n_q_heads);
                    const __half *q = static_cast<const __half *>(a.q) +
                                      (row < 0 ? 0 : (t.start[ahead.b] + token) * a.q_stride + head * D) + c * 16;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        copy16(dst + S::kQ + (nt * (D / 32) + i) * 512 + lane * 16, q + (i >> 1) * 64 + (i & 1) * 8,
                               row < 0 ? 0 : 16);
                }
            }
            ++pu;
            pfirst = ahead.next(t, a, kRows, group);
            pstage = pstage + 1 == S::kStages ? 0 : pstage + 1;
        }
        commit();
    };

    if (lane == 0) pieces[2 * warp].slot = pieces[2 * warp + 1].slot = -1;
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) copy_next();

    Segment seg;
    if (u0 < u1) seg.find(t, a, kRows, group, u0);
    int stage = 0;
    for (int u = u0; u < u1;) {
        // --- a piece of a segment: units u to end
        const int seg_first = seg.first(u), seg_end = seg_first + seg.tiles, end = min(seg_end, u1);
        const int L = len[seg.b], n = start[seg.b + 1] - start[seg.b];
        uint32_t q[NT][D / 16][2];
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
                limit[nt][i] = L - n + 1 + min((seg.rt * kRows + nt * 8 + 2 * c + i) / group, n - 1);
            }
        }
        const int least = L - n + 1 + seg.rt * kRows / group;  // of the tile's first row
        float w = 0.f, inv_w = 0.f;
        bool first = true;
        for (; u < end; ++u) {
            wait_copies<S::kStages - 2>();
            copy_next();  // into the stage read last time
            const unsigned char *p = ring_p + stage * S::kStage;
            stage = stage + 1 == S::kStages ? 0 : stage + 1;
            if (first) {
                first = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(
                            p + S::kQ + (nt * (D / 32) + i) * 512 + lane * 16);
                        q[nt][2 * i][0] = x.x;
                        q[nt][2 * i][1] = x.y;
                        q[nt][2 * i + 1][0] = x.z;
                        q[nt][2 * i + 1][1] = x.w;
                    }
            }
            const int tok = (u - seg_first) * kTile;
            const float2 scales = *reinterpret_cast<const float2 *>(p + S::kS + lane * 8);
            const float f = scales.x * a.scale_log2;
            // --- scores
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {
                const uint4 x = *reinterpret_cast<const uint4 *>(p + (2 * half) * 512 + lane * 16);
                const uint4 y = *reinterpret_cast<const uint4 *>(p + (2 * half + 1) * 512 + lane * 16);
                const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t frag[4] = {q8_widen<KIND, 0>(wx[i]), q8_widen<KIND, 0>(wy[i]),
                                              q8_widen<KIND, 1>(wx[i]), q8_widen<KIND, 1>(wy[i])};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_16816(s[nt], frag, q[nt][half * 4 + i][0], q[nt][half * 4 + i][1]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[nt][i] *= f;
            if (tok + kTile > least) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (tok + r + (i >> 1) * 8 >= limit[nt][i & 1]) s[nt][i] = -INFINITY;
            }
            // --- references
            bool move = scales.y > 0.f && !(scales.y >= w * (1.f / 64.f) && scales.y <= w * 16.f);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) move = move || s[nt][i] > m[nt][i & 1] + kMoveM;
            if (__any_sync(~0u, move)) {
                float g = 1.f;
                if (scales.y > 0.f && !(scales.y >= w * (1.f / 64.f) && scales.y <= w * 16.f)) {
                    inv_w = __fdividef(1.f, scales.y);
                    g = w * inv_w;
                    w = scales.y;
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
            const float fv = scales.y * inv_w;
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
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(p + S::kV + i * 512 + lane * 16);
                    v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(p + S::kV + i * 256 + lane * 8);
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
                    const long long row = row_at(t, a, seg, kRows, group, nt * 8 + 2 * c + i, &token);
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
            // the range's first piece has a record of its own; a later one is the last
            // thing the warp does, and takes the ring
            const int slot = seg_first < u0 ? 0 : 1;
            if (slot == 1) wait_copies<0>();
            __syncwarp();
            float *rec = slot ? reinterpret_cast<float *>(ring_p) : records + warp * S::kRecord;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = nt * 8 + 2 * c + i;
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt)
                        *reinterpret_cast<float2 *>(rec + row * D + r * S::kVPiece + 2 * mt) =
                            make_float2(o[nt][mt][i] * w, o[nt][mt][i + 2] * w);
                    if (r == 0) {
                        rec[kRows * D + row] = m[nt][i];
                        rec[kRows * D + kRows + row] = l[nt][i];
                    }
                }
            if (lane == 0) pieces[2 * warp + slot] = Piece{seg_first, seg_end, slot, seg};
        }
        if (u < u1) {
            seg.j = seg.tiles - 1;
            seg.next(t, a, kRows, group);
        }
    }
    wait_copies<0>();
    __syncthreads();

    // --- joins: runs of pieces of one segment, in the order of the warps
    unsigned char *ws = static_cast<unsigned char *>(a.workspace);
    int *counters = reinterpret_cast<int *>(ws);
    float *parts = reinterpret_cast<float *>(ws + kBalancedCounterBytes);
    Piece open[2];  // this CTA's parts of segments that other CTAs share
    open[0].slot = open[1].slot = -1;
    for (int i = 0; i < 2 * kWarps;) {
        if (pieces[i].slot < 0) {
            ++i;
            continue;
        }
        const Piece head = pieces[i];
        int e = i + 1;
        while (e < 2 * kWarps && (pieces[e].slot < 0 || pieces[e].first == head.first)) ++e;
        const bool whole = head.first >= U0 && head.end <= U1;
        const int side = head.first >= U0 ? 1 : 0;
        float *part = parts + (static_cast<long long>(cta) * 2 + side) * S::kRecord;
        if (!whole) open[side] = head;
        for (int x = threadIdx.x; x < kRows * D / 4; x += kWarps * 32) {
            const int row = x / (D / 4);
            float top = -INFINITY;
            for (int k = i; k < e; ++k)
                if (pieces[k].slot >= 0) {
                    const float *rec = pieces[k].slot ? reinterpret_cast<const float *>(smem + (k / 2) * S::kStages * S::kStage)
                                                      : records + (k / 2) * S::kRecord;
                    top = fmaxf(top, rec[kRows * D + row]);
                }
            const float ref = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = i; k < e; ++k)
                if (pieces[k].slot >= 0) {
                    const float *rec = pieces[k].slot ? reinterpret_cast<const float *>(smem + (k / 2) * S::kStages * S::kStage)
                                                      : records + (k / 2) * S::kRecord;
                    const float g = ex2(rec[kRows * D + row] - ref);
                    const float4 y = reinterpret_cast<const float4 *>(rec)[x];
                    sum += g * rec[kRows * D + kRows + row];
                    acc.x += g * y.x;
                    acc.y += g * y.y;
                    acc.z += g * y.z;
                    acc.w += g * y.w;
                }
            if (whole) {
                int token;
                const long long at_row = row_at(t, a, head.at, kRows, group, row, &token);
                if (at_row >= 0) {
                    const float z = 1.f / sum;
                    uint2 y = make_uint2(pack_half2(acc.x * z, acc.y * z), pack_half2(acc.z * z, acc.w * z));
                    reinterpret_cast<uint2 *>(a.out)[at_row * (D / 4) + x % (D / 4)] = y;
                    if (a.lse_out && x % (D / 4) == 0) a.lse_out[at_row] = (top + log2f(sum)) * kLn2;
                }
            } else {
                reinterpret_cast<float4 *>(part)[x] = acc;
                if (x % (D / 4) == 0) {
                    part[kRows * D + row] = top;
                    part[kRows * D + kRows + row] = sum;
                }
            }
        }
        i = e;
    }
    // --- segments of several CTAs: the last to arrive joins
    if (open[0].slot < 0 && open[1].slot < 0) return;
    auto owner = [&](int u) { return static_cast<int>((static_cast<long long>(u + 1) * ctas - 1) / total); };
    __threadfence();
    __syncthreads();
    if (threadIdx.x < 2) {
        const int side = threadIdx.x;
        last_of[side] = 0;
        if (open[side].slot >= 0) {
            const int from = owner(open[side].first), more = owner(open[side].end - 1) - from;
            const int old = atomic_add_acq_rel_gpu(counters + from, 1);
            if (counter_not_zeroed(old, more)) {
                flag_error(a.err, PKV_ERRBIT_WORKSPACE);
                atomic_exch_relaxed_gpu(counters + from, kCounterPoison);
            } else if (old == more) {
                last_of[side] = 1;
                red_add_relaxed_gpu(counters + from, -(more + 1));
            }
        }
    }
    __syncthreads();
    for (int side = 0; side < 2; ++side) {
        if (!last_of[side]) continue;
        __threadfence();
        const Piece &head = open[side];
        const int from = owner(head.first), to = owner(head.end - 1);
        for (int x = threadIdx.x; x < kRows * D / 4; x += kWarps * 32) {
            const int row = x / (D / 4);
            int token;
            const long long at_row = row_at(t, a, head.at, kRows, group, row, &token);
            if (at_row < 0) continue;
            float top = -INFINITY;
            for (int k = from; k <= to; ++k)
                top = fmaxf(top, __ldcg(parts + (2ll * k + (k == from)) * S::kRecord + kRows * D + row));
            const float ref = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = from; k <= to; ++k) {
                const float *rec = parts + (2ll * k + (k == from)) * S::kRecord;
                const float g = ex2(__ldcg(rec + kRows * D + row) - ref);
                const float4 y = __ldcg(reinterpret_cast<const float4 *>(rec) + x);
                sum += g * __ldcg(rec + kRows * D + kRows + row);
                acc.x += g * y.x;
                acc.y += g * y.y;
                acc.z += g * y.z;
                acc.w += g * y.w;
            }
            const float z = 1.f / sum;
            uint2 y = make_uint2(pack_half2(acc.x * z, acc.y * z), pack_half2(acc.z * z, acc.w * z));
            reinterpret_cast<uint2 *>(a.out)[at_row * (D / 4) + x % (D / 4)] = y;
            if (a.lse_out && x % (D / 4) == 0) a.lse_out[at_row] = (top + log2f(sum)) * kLn2;
        }
    }
}

template <int KIND, int D, int NT>
cudaError_t launch(const Q8AttentionArgs &a, const Q8Split &sp, cudaStream_t stream) {
    const size_t smem = Shape<D, NT>::smem(a.num_seqs);
    const cudaError_t e = cudaFuncSetAttribute(q8_attention_kernel<KIND, D, NT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_pdl(q8_attention_kernel<KIND, D, NT>, dim3(sp.ctas), dim3(kWarps * 32), smem, stream, a);
}

template <int KIND, int D>
cudaError_t launch_rows(const Q8AttentionArgs &a, const Q8Split &sp, cudaStream_t stream) {
    return sp.row_tiles == 1 ? launch<KIND, D, 1>(a, sp, stream) : launch<KIND, D, 2>(a, sp, stream);
}

static_assert(Shape<128, 1>::smem(kQ8MaxSeqs) <= 227 * 1024 - 2048, "shared memory");
static_assert(Shape<128, 2>::smem(kQ8MaxSeqs) <= 227 * 1024 - 2048, "shared memory");

}  // namespace

bool q8_split(int num_seqs, int max_q_len, int n_q_heads, int n_kv_heads, int head_dim, int max_len,
              int sms, Q8Split *sp) {
    const long long rows = static_cast<long long>(max_q_len) * (n_q_heads / n_kv_heads);
    sp->row_tiles = rows <= 8 ? 1 : 2;
    const long long height = 8 * sp->row_tiles;
    const long long tiles = (static_cast<long long>(max_len) + kTile - 1) / kTile;
    const double units = static_cast<double>(num_seqs) * n_kv_heads * tiles * ((rows + height - 1) / height);
    if (units >= 2147483648.0) return false;
    sp->ctas = sms;
    if (static_cast<size_t>(sms) * 4 > kBalancedCounterBytes) sp->ctas = kBalancedCounterBytes / 4;
    const size_t record = (height * head_dim + 2 * height) * 4;
    sp->ws_bytes = kBalancedCounterBytes + static_cast<size_t>(sp->ctas) * 2 * record;
    return true;
}

cudaError_t launch_q8_attention(const Q8AttentionArgs &a, int kind, const Q8Split &sp,
                                cudaStream_t stream) {
    if (a.head_dim == 128)
        return kind == PKV_Q8_E4M3 ? launch_rows<PKV_Q8_E4M3, 128>(a, sp, stream)
                                   : launch_rows<PKV_Q8_INT8, 128>(a, sp, stream);
    return kind == PKV_Q8_E4M3 ? launch_rows<PKV_Q8_E4M3, 64>(a, sp, stream)
                               : launch_rows<PKV_Q8_INT8, 64>(a, sp, stream);
}

}  // namespace pkv
