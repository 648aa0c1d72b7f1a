// latent_prefill.cu -- expanded latent attention of prompts
// (latent_prefill_attention): causal attention with keys [k, k_rope] of D + 64
// entries and values of D.
//
// For a tile of 128 query rows and a step of 96 keys
//   S [128 x 96] = Q [k, k_rope]^T         12 products of 16 entries (D = 128)
//   P = 2^(S scale - r), r per row; O (+)= P V    6 products of 16 keys
// with S, O and P in TMEM: P (fp16) takes the place of its own S and is the first
// operand of the second product, so it never passes through shared memory.  r is the
// running maximum, less kHead, and moves only when a score is far above it; O is then
// rescaled in TMEM by the thread that owns the row.
//
// A CTA has two neighbouring tiles, which share the keys and values that TMA copies
// bring: one tile's softmax (a warpgroup, a row a thread) runs under the other's
// products.  Bound by the chain of one tile: products 1070 cycles (57 per 96-wide
// score product: its operands' shared-memory reads, 64 per output product), signal
// and wait 430, softmax 1100; a step of both tiles takes about 2500 cycles, of which
// 2140 are products.  4096 tokens x 128 heads: 538 us in calls one after another, 1277
// TFLOP/s (66 % of what a large bf16 matrix product reaches in a burst); 503 us behind
// less work (six calls in a graph): the clock follows the power drawn before.
//
// P is fp16 because the values, the other operand of its product, are: half a step of
// each weight, 2^-11, as much as the result's own rounding.  The row sums take the
// weights before that rounding; they, the references and O are fp32, and so are the
// parts that a cluster joins.
//
// Where there are few items, a cluster of two or four CTAs has one, each a part of its
// keys, and joins the parts through shared memory.
//
// Why 96 keys a step: two steps of keys and values (2 x 60 KB) fit beside the two
// tiles' queries (96 KB); with 128 there is room for one and a half, and the values
// of a step would come a copy's latency late.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>

#include "pagedkv_latent.h"
#include "pkv_internal.h"
#include "rope_latent.h"
#include "tc05.cuh"

namespace pkv {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

namespace {

constexpr int kP = 64;          // rotated entries
constexpr int kRows = 128;      // query rows of a tile
constexpr int kKeys = 96;       // key rows of a step
constexpr int kThreads = 384;   // two softmax warpgroups; copy warp, two MMA warps, an idle one
// Registers move from the third warpgroup to the softmax: 8 x 32 x 208 + 4 x 32 x 88
// is the 12 x 32 x 168 of the launch.
constexpr int kQPlane = kRows * 128, kKPlane = kKeys * 128;  // 64 columns of a tile, bytes
// P holds 2^(s - r) with r kHead below the running maximum: weights up to
// 2^kHead, and up to 2^(kHead + kLag) before r follows; fp16 ends at 2^16.
constexpr float kHead = 6.f, kLag = 8.f;

template <int D>
struct Cfg {
    static constexpr int KP = D / 64 + 1, VP = D / 64;  // planes of 64 columns
    static constexpr int STAGES = D == 128 ? 2 : 4;
    static constexpr int Q_BYTES = 2 * KP * kQPlane;
    static constexpr int STAGE_BYTES = (KP + VP) * kKPlane;
    static constexpr int SMEM = 1024 + Q_BYTES + STAGES * STAGE_BYTES;
};

struct Shared {
    uint64_t q_full[2], q_empty[2], s_full[2], p_ready[2][2], o_done[2], o_free[2];
    uint64_t full[4], empty[4], item_full[2], item_free[2], answered, turn[2], drained[2];
    uint4 answer;   // of the hardware, to the copy role
    uint4 item[2];  // of the copy role, to the others: a CTA's coordinates, 1; or 0 at the end
    uint32_t tmem;
    int stop;
    // what the copy role issued: pairs of keys and values, query tiles, and whether (and
    // which) an answer of the hardware is still to come
    int begun, queries[2], awaited, answers;
};

// One CTA's worth of work: two neighbouring tiles of query rows of one head and, in a
// cluster of CL CTAs, this CTA's part of their key steps.
struct Item {
    int h, pair, q0, n, k0, m;
    int steps[2], total;  // key steps of the tiles, and of both
    int whole, first;     // those of the whole cluster; the first key of this CTA's
};

// The work of CTA `cta`; false when it has none.
template <int CL>
__device__ __forceinline__ bool load_item(const LatentPrefillArgs &a, const uint3 &cta, bool tell,
                                          Item *it) {
    const int seq = cta.z;
    it->h = cta.y;
    it->pair = (gridDim.x - 1 - cta.x) / CL;  // the longest rows first
    it->whole = it->first = 0;
    it->q0 = a.q_start[seq];
    it->n = a.q_start[seq + 1] - it->q0;
    it->k0 = a.kv_start[seq];
    it->m = a.kv_start[seq + 1] - it->k0;
    if (it->n == 0) return false;
    if (it->n < 0 || it->n > it->m || it->n > a.max_q_len || it->m > a.max_kv_len || it->q0 < 0 ||
        it->k0 < 0 || it->n > a.total_q - it->q0 || it->m > a.total_kv - it->k0) {
        if (tell) flag_error(a.err, PKV_ERRBIT_CONTEXT);
        return false;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = (2 * it->pair + t) * kRows;
        const int last = min(first + kRows, it->n) - 1;
        it->steps[t] = first < it->n ? (it->m - it->n + last + kKeys) / kKeys : 0;
    }
    it->whole = it->total = max(it->steps[0], it->steps[1]);
    if (CL > 1) {
        const int rank = cta.x % CL, from = it->whole * rank / CL;
        it->total = it->whole * (rank + 1) / CL - from;
#pragma unroll
        for (int t = 0; t < 2; ++t) it->steps[t] = min(max(it->steps[t] - from, 0), it->total);
        it->first = from * kKeys;
    }
    return it->total > 0;
}

// The copy role finds the items that have work: its own CTA's, then those of CTAs
// not launched yet, which it takes over.  It hands them to the other roles through two
// places; a place is free again when all ten readers have read it.
struct Items {
    int k;  // items read

    // The next item, or false at the end (or when the kernel gives up).
    template <int CL>
    __device__ bool advance(const LatentPrefillArgs &a, Shared &sh, bool whole_warp, Item *it) {
        volatile int *stop = &sh.stop;
        const int s = k & 1;
        const bool ok = whole_warp ? warp_wait_or_stop(&sh.item_full[s], (k >> 1) & 1, stop)
                                   : wait_or_stop(&sh.item_full[s], (k >> 1) & 1, stop);
        if (!ok) return false;
        const uint4 c = sh.item[s];
        ++k;
        if (whole_warp) __syncwarp();
        if (!whole_warp || (threadIdx.x & 31) == 0) mbar_arrive(&sh.item_free[s]);
        return c.w != 0 && load_item<CL>(a, make_uint3(c.x, c.y, c.z), false, it);
    }
};

// The CTAs of a cluster have attended a part of the keys each; CTA c finishes the columns
// [c D / CL, (c + 1) D / CL) of both tiles.  Every CTA sends the others its rows'
// references and sums and their columns of O, into the memory of the ring (whose copies
// and products are over at the first barrier); `part`: this warp's tile had a step.
template <int D, int CL>
__device__ __forceinline__ void join_parts(const LatentPrefillArgs &a, const Item &it,
                                           unsigned char *ring, uint32_t to, bool part, float r,
                                           float l) {
    constexpr int W = D / CL;  // columns of a CTA
    static_assert(CL * 2048 + (CL - 1) * W * 1024 <= Cfg<D>::STAGES * Cfg<D>::STAGE_BYTES, "in the ring");
    const uint32_t rank = cluster_rank();
    const int row = threadIdx.x;  // of the 256 of both tiles
    const bool some = part && l != 0.f;
    const uint32_t stats = smem_addr(ring), parts = stats + CL * 2048;
    __syncwarp();
    cluster_sync();
    if (it.whole > 0) {
#pragma unroll
        for (int x = 1; x <= CL; ++x) {
            const uint32_t c = (rank + x) % CL;
            store_peer2(peer_addr(stats + (rank * 256 + row) * 8, c), some ? r : -INFINITY,
                        part ? l : 0.f);
            if (x == CL || !part) continue;
            // CTA c finds this one's columns in place x - 1
            const uint32_t dst = peer_addr(parts + ((x - 1) * (W / 4) * 256 + row) * 16, c);
#pragma unroll
            for (int v = 0; v < W; v += 16) {
                uint32_t o[16];
                tmem_ld16(o, to + c * W + v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 4; ++e) store_peer4(dst + (v / 4 + e) * 4096, o + 4 * e);
            }
        }
    }
    __syncwarp();
    cluster_sync();
    const int i = 2 * kRows * it.pair + row;  // of the sequence's queries
    if (it.whole == 0) return;
    float2 st[CL];  // of the CTAs rank, rank - 1, rank - 2 ..
    float top = -INFINITY, sum = 0.f, f[CL];
#pragma unroll
    for (int x = 0; x < CL; ++x) {
        st[x] = *reinterpret_cast<const float2 *>(ring + (((rank + CL - x) % CL) * 256 + row) * 8);
        top = fmaxf(top, st[x].x);
    }
#pragma unroll
    for (int x = 0; x < CL; ++x) {
        f[x] = st[x].y == 0.f ? 0.f : ex2(st[x].x - top);
        sum += st[x].y * f[x];
    }
    const float inv = 1.f / sum;
    const long long at = static_cast<long long>(it.q0 + i) * a.n_heads + it.h;
    uint4 *out = reinterpret_cast<uint4 *>(static_cast<__half *>(a.out) + at * D + rank * W);
    const float4 *others = reinterpret_cast<const float4 *>(ring + CL * 2048) + row;
#pragma unroll
    for (int v = 0; v < W; v += 16) {
        float y[16];
        uint32_t o[16];
        if (part) {
            tmem_ld16(o, to + rank * W + v);
            tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = f[0] != 0.f ? __uint_as_float(o[e]) * f[0] : 0.f;
#pragma unroll
        for (int x = 1; x < CL; ++x) {
            if (f[x] == 0.f) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 z = others[((x - 1) * (W / 4) + v / 4 + e) * 256];
                y[4 * e] += z.x * f[x];
                y[4 * e + 1] += z.y * f[x];
                y[4 * e + 2] += z.z * f[x];
                y[4 * e + 3] += z.w * f[x];
            }
        }
        if (i < it.n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = pack_half2(y[8 * e + 2 * k] * inv, y[8 * e + 2 * k + 1] * inv);
                out[v / 8 + e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    if (rank == 0 && a.lse_out && i < it.n) a.lse_out[at] = (top + log2f(sum)) * 0.69314718055994531f;
}

template <int D, int CL>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const LatentPrefillArgs a, const __grid_constant__ CUtensorMap mq,
                          const __grid_constant__ CUtensorMap mkv,
                          const __grid_constant__ CUtensorMap mr) {
    using C = Cfg<D>;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(16) Shared sh;
    unsigned char *base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sh.q_full[t], 1);
            mbar_init(&sh.q_empty[t], 1);
            mbar_init(&sh.s_full[t], 1);
            mbar_init(&sh.p_ready[t][0], 4);
            mbar_init(&sh.p_ready[t][1], 4);
            mbar_init(&sh.o_done[t], 1);
            mbar_init(&sh.o_free[t], 4);
            mbar_init(&sh.item_full[t], 1);
            mbar_init(&sh.item_free[t], 10);  // eight warps and two threads
            mbar_init(&sh.drained[t], 1);
            mbar_init(&sh.turn[t], 1);
        }
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 2);
        }
        mbar_init(&sh.answered, 1);
        sh.stop = sh.begun = sh.queries[0] = sh.queries[1] = sh.awaited = 0;
        fence_barrier_init();
    }
    if (warp == 9) tmem_alloc(&sh.tmem, 512);
    if (warp == 8 && lane == 0) {
        prefetch_tmap(&mq);
        prefetch_tmap(&mkv);
        prefetch_tmap(&mr);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dependency_wait();
    allow_dependent_launch();
    const uint32_t tmem = sh.tmem;
    volatile int *stop = &sh.stop;
    Items items{0};
    Item it;
    // TMEM columns: S of tile t at 128 t (P in its first half), O at 256 + 128 t

    if (warp >= 8) {
    give_registers<88>();
    if (warp == 8) {
        // --- copies ---
        if (elect_one()) {
            // Pair f of the ring is the keys of step f and the values of step f - 1:
            // what the products between two softmax steps take, on one barrier.
            // Steps count on over the items.
            int f = 0;
            int q[2] = {0, 0};  // query tiles so far
            bool ok = true, open = CL == 1;  // open: the hardware may have more CTAs
            int answers = 0, handed = 0;
            Item last;        // whose final values are still to come
            auto ask = [&] {  // for the CTA after the one at hand
                mbar_arrive_expect_tx(&sh.answered, 16);
                ask_next_cta(&sh.answer, &sh.answered);
            };
            uint3 cta = blockIdx;
            // hands on the item of `cta`, or of the first CTA after it that has one;
            // the next answer is then under way
            auto hand_on = [&] {
                bool have = load_item<CL>(a, cta, true, &it);
                while (ok && !have && open) {
                    ok = wait_or_stop(&sh.answered, answers & 1, stop);
                    if (!ok) break;
                    ++answers;
                    open = next_cta(&sh.answer, &cta);
                    fence_proxy_async_smem();
                    if (open) {
                        ask();
                        have = load_item<CL>(a, cta, true, &it);
                    }
                }
                const int s = handed & 1;
                ok = ok && wait_or_stop(&sh.item_free[s], ((handed >> 1) & 1) ^ 1, stop);
                if (!ok) return false;
                sh.item[s] = make_uint4(cta.x, cta.y, cta.z, have ? 1 : 0);
                mbar_arrive(&sh.item_full[s]);
                ++handed;
                return have;
            };
            // the next pair: values of vi at step vj, keys of ki at step kj (either null)
            auto copy_pair = [&](const Item *vi, int vj, const Item *ki, int kj) {
                const int s = f % C::STAGES;
                ok = wait_or_stop(&sh.empty[s], ((f / C::STAGES) & 1) ^ 1, stop);
                if (!ok) return;
                mbar_arrive_expect_tx(&sh.full[s], (ki ? C::KP * kKPlane : 0) + (vi ? C::VP * kKPlane : 0));
                unsigned char *st = base + C::Q_BYTES;
                if (vi)
#pragma unroll 1
                    for (int p = 0; p < C::VP; ++p)
                        tma_load_3d(st + ((f - 1) % C::STAGES) * C::STAGE_BYTES + (C::KP + p) * kKPlane,
                                    &mkv, D + 64 * p, vi->h, vi->k0 + vi->first + vj * kKeys, &sh.full[s]);
                if (ki) {
#pragma unroll 1
                    for (int p = 0; p < D / 64; ++p)
                        tma_load_3d(st + s * C::STAGE_BYTES + p * kKPlane, &mkv, 64 * p, ki->h,
                                    ki->k0 + ki->first + kj * kKeys, &sh.full[s]);
                    tma_load_2d(st + s * C::STAGE_BYTES + (D / 64) * kKPlane, &mr, 0,
                                ki->k0 + ki->first + kj * kKeys, &sh.full[s]);
                }
                ++f;
            };
            if (open) ask();
            bool have = hand_on();
            while (ok && have) {
#pragma unroll 1
                for (int j = 0; j < it.total && ok; ++j) {
                    copy_pair(j > 0 ? &it : f > 0 ? &last : nullptr, j > 0 ? j - 1 : last.total - 1,
                              &it, j);
                    if (j == 0)
#pragma unroll 1
                        for (int t = 0; t < 2 && ok; ++t)
                            if (it.steps[t] > 0) {
                                ok = wait_or_stop(&sh.q_empty[t], (q[t] & 1) ^ 1, stop);
                                if (!ok) break;
                                ++q[t];
                                mbar_arrive_expect_tx(&sh.q_full[t], C::KP * kQPlane);
                                for (int p = 0; p < C::KP; ++p)
                                    tma_load_3d(base + (t * C::KP + p) * kQPlane, &mq, 64 * p,
                                                it.h, it.q0 + (2 * it.pair + t) * kRows,
                                                &sh.q_full[t]);
                            }
                }
                if (!ok) break;
                last = it;
                if (open) {
                    // the answer asked for while this item's copies were issued
                    ok = wait_or_stop(&sh.answered, answers & 1, stop);
                    if (!ok) break;
                    ++answers;
                    open = next_cta(&sh.answer, &cta);
                    fence_proxy_async_smem();
                    if (open) ask();
                }
                if (open) {
                    have = hand_on();
                } else {
                    have = false;
                    const int s = handed & 1;
                    ok = wait_or_stop(&sh.item_free[s], ((handed >> 1) & 1) ^ 1, stop);
                    if (!ok) break;
                    sh.item[s] = make_uint4(0, 0, 0, 0);
                    mbar_arrive(&sh.item_full[s]);
                    ++handed;
                }
            }
            if (ok && f > 0) copy_pair(&last, last.total - 1, nullptr, 0);
            sh.begun = f;
            sh.queries[0] = q[0];
            sh.queries[1] = q[1];
            sh.awaited = !ok && open;
            sh.answers = answers;
        }
    } else if (warp < 11) {
        // --- matrix products ---
        // One warp a tile, in turns of the products between two of the tile's softmax
        // steps: a warp's waits and commits pass while the other's products run, and
        // one tile's softmax runs under the other's products.  (One thread for both
        // tiles left the tensor core idle for 1240 of a step's 3400 cycles: it takes
        // hardly more than the next product ahead of time.  Without turns the two
        // tiles fall into step, and nothing runs under their softmax: 3600.)
        if (elect_one()) {
            const int t = warp - 9;
            constexpr uint32_t ds = mma_desc(kRows, kKeys, false, false);
            constexpr uint32_t dpv = mma_desc(kRows, D, false, true);
            const uint32_t kv_addr = smem_addr(base) + C::Q_BYTES, ts = tmem + 128 * t;
            const uint64_t qd = smem_desc(smem_addr(base) + t * C::KP * kQPlane, 1024, 0);
            int f = 0;       // key steps so far
            int sc = 0, qc = 0;  // this tile's steps and items
            int turns = 0;
            bool more = items.advance<CL>(a, sh, false, &it);
            bool ok = !more || first_wait(&sh.full[0], 0, a.first_wait_polls, stop);
            int steps = 0, total = 0;  // of the item at hand
            int j = -1;  // its step whose weights come next; -1: only the first scores
            while (ok) {
                // between the softmax of step j and that of the step after it, which is
                // step j + 1 of the item or the first of the next one
                const bool end = j + 1 == total;
                if (end && j >= 0) more = items.advance<CL>(a, sh, false, &it);
                if (j < 0 && !more) break;
                const int pair = j < 0 ? f : f + 1;  // of copies; also the step of its keys
                ok = wait_or_stop(&sh.full[pair % C::STAGES], (pair / C::STAGES) & 1, stop);
                const bool weights = j >= 0 && j < steps;
                if (ok && weights) {
                    if (j == 0) ok = wait_or_stop(&sh.o_free[t], qc & 1, stop);
                    ok = ok && wait_or_stop(&sh.p_ready[t][0], sc & 1, stop);
                }
                ok = ok && wait_or_stop(&sh.turn[t], (turns & 1) ^ (t ^ 1), stop);
                if (!ok) break;
                ++turns;
                tc_fence_after();
                if (weights) {
                    const uint64_t vd = smem_desc(kv_addr + (f % C::STAGES) * C::STAGE_BYTES +
                                                      C::KP * kKPlane, 1024, kKPlane);
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        mma_ts(ts + 256, ts + 8 * k, vd + k * 128, dpv, j > 0 || k > 0);
                    ok = wait_or_stop(&sh.p_ready[t][1], sc & 1, stop);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 3; k < 6; ++k) mma_ts(ts + 256, ts + 8 * k, vd + k * 128, dpv, true);
                    ++sc;
                    if (j + 1 == steps) mma_commit(&sh.o_done[t]);
                }
                const int next_steps = more ? it.steps[t] : 0;
                const bool first = end && next_steps > 0;
                if (j + 1 < steps || first) {
                    if (first) {
                        ok = wait_or_stop(&sh.q_full[t], qc & 1, stop);
                        if (!ok) break;
                        ++qc;
                    }
                    tc_fence_after();
                    const uint64_t kd = smem_desc(kv_addr + (pair % C::STAGES) * C::STAGE_BYTES, 1024, 0);
#pragma unroll
                    for (int k = 0; k < 4 * C::KP; ++k)
                        mma_ss(ts, qd + (k / 4) * (kQPlane / 16) + (k % 4) * 2,
                               kd + (k / 4) * (kKPlane / 16) + (k % 4) * 2, ds, k > 0);
                    mbar_arrive(&sh.turn[t ^ 1]);
                    mma_commit(&sh.s_full[t]);
                    if (first ? next_steps == 1 : j + 2 == steps) mma_commit(&sh.q_empty[t]);
                } else {
                    mbar_arrive(&sh.turn[t ^ 1]);
                }
                mma_commit(&sh.empty[pair % C::STAGES]);
                if (j >= 0) ++f;
                ++j;
                if (end) {
                    if (!more) break;
                    steps = next_steps;
                    total = it.total;
                    j = 0;
                }
            }
            // nothing of the tensor core is left in flight when TMEM is freed
            mma_commit(&sh.drained[t]);
            mbar_wait_bounded(&sh.drained[t], 0);
        }
    }
    } else {
        // --- softmax, results ---
        take_registers<208>();
        const int t = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 * (warp % 4) << 16
        const uint32_t ts = tmem + 128 * t + lanes, to = tmem + 256 + 128 * t + lanes;
        const float scale = a.scale_log2;
        int f = 0, sc = 0, mine = 0;  // key steps, this tile's, and its items so far
        bool have = items.advance<CL>(a, sh, true, &it);
        bool ok = true;
        float r = 0.f, l = 0.f;
        while (have) {
            const int i = (2 * it.pair + t) * kRows + (threadIdx.x & 127);
            const int seen = min(it.m - it.n + i + 1, it.m);  // keys this row attends
            r = l = 0.f;
            for (int j = 0; j < it.steps[t]; ++j, ++sc) {
                ok = warp_wait_or_stop(&sh.s_full[t], sc & 1, stop);
                if (!ok) break;
                tc_fence_after();
                uint32_t sb[3][32];
#pragma unroll
                for (int c = 0; c < 3; ++c) tmem_ld32(sb[c], ts + 32 * c);
                tmem_wait_ld();
                float x[kKeys];
#pragma unroll
                for (int c = 0; c < kKeys; ++c) x[c] = __uint_as_float(sb[c / 32][c % 32]);
                if (a.negate) {
#pragma unroll
                    for (int c = 0; c < kKeys; ++c) x[c] = -x[c];
                }
                const int left = seen - it.first - j * kKeys;
                if (__any_sync(0xffffffffu, left < kKeys)) {
#pragma unroll
                    for (int c = 0; c < kKeys; ++c) x[c] = c < left ? x[c] : -INFINITY;
                }
                float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int c = 4; c + 1 < kKeys; c += 2)
                    mx[(c / 2) & 3] = max3(mx[(c / 2) & 3], x[c], x[c + 1]);
                const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * scale;
                if (j == 0) {
                    r = top > -INFINITY ? top - kHead : 0.f;
                } else {
                    const bool move = top - r > kHead + kLag;
                    if (__any_sync(0xffffffffu, move)) {
                        // O follows the new reference; S being full, every earlier
                        // product into O is done
                        const float next = move ? top - kHead : r;
                        const float fac = ex2(r - next);
                        r = next;
                        l *= fac;
#pragma unroll
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(o, to + c);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * fac);
                            tmem_st32(to + c, o);
                        }
                    }
                }
                // values of rows beyond the sequence's keys meet weights of 0: they
                // must be finite, so the last step's are cleared
                const int valid = it.m - it.first - j * kKeys;
                if (valid < kKeys) {
                    const int s = (f + j) % C::STAGES, pair = f + j + 1;
                    ok = warp_wait_or_stop(&sh.full[pair % C::STAGES], (pair / C::STAGES) & 1, stop);
                    if (!ok) break;
                    unsigned char *v = base + C::Q_BYTES + s * C::STAGE_BYTES + C::KP * kKPlane;
                    const int pieces = (kKeys - valid) * 8;
                    for (int e = threadIdx.x & 127; e < pieces * C::VP; e += 128)
                        *reinterpret_cast<uint4 *>(v + (e / pieces) * kKPlane + valid * 128 +
                                                   (e % pieces) * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t p16[16], p8[8];
#pragma unroll
                    for (int c = 0; c < 24; ++c) {
                        const float2 e = fma2(make_float2(x[half * 48 + 2 * c], x[half * 48 + 2 * c + 1]),
                                              scale, -r);
                        const float y0 = ex2(e.x), y1 = ex2(e.y);
                        sum[c & 1] = add2(sum[c & 1], make_float2(y0, y1));
                        if (c < 16) p16[c] = pack_half2(y0, y1); else p8[c - 16] = pack_half2(y0, y1);
                    }
                    tmem_st16(ts + half * 24, p16);
                    tmem_st8(ts + half * 24 + 16, p8);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.p_ready[t][half]);
                }
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
            }
            if (!ok) break;
            if (it.steps[t] > 0) {
                ok = warp_wait_or_stop(&sh.o_done[t], mine & 1, stop);
                if (!ok) break;
                ++mine;
                tc_fence_after();
                if (CL > 1) break;  // the parts are joined below
                const float inv = 1.f / l;
                const long long row = static_cast<long long>(it.q0 + i) * a.n_heads + it.h;
                uint4 *out = reinterpret_cast<uint4 *>(static_cast<__half *>(a.out) + row * D);
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(o, to + c);
                    tmem_wait_ld();
                    if (c + 32 == D) {
                        // the next item's products may write O
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.o_free[t]);
                    }
                    if (i < it.n) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                w[k] = pack_half2(__uint_as_float(o[8 * e + 2 * k]) * inv,
                                                  __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                            out[c / 8 + e] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                if (a.lse_out && i < it.n) a.lse_out[row] = (r + log2f(l)) * 0.69314718055994531f;
            }
            if (CL > 1) break;
            f += it.total;
            have = items.advance<CL>(a, sh, true, &it);
        }
        if constexpr (CL > 1) {
            const bool part = have && ok && it.steps[t] > 0;
            load_item<CL>(a, blockIdx, false, &it);
            join_parts<D, CL>(a, it, base + C::Q_BYTES, to, part, r, l);
        }
    }
    if (CL > 1 && warp >= 8) {  // the two barriers of join_parts
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && sh.stop) {
        flag_error(a.err, PKV_ERRBIT_TIMEOUT);
        // Every copy in flight lands before the CTA gives its memory back.  Not until here:
        // the copy role may have issued its last one before another role gave up.
        for (int t = 0; t < 2; ++t)
            if (sh.queries[t] > 0) mbar_wait_bounded(&sh.q_full[t], (sh.queries[t] - 1) & 1);
        for (int i = max(0, sh.begun - C::STAGES); i < sh.begun; ++i)
            mbar_wait_bounded(&sh.full[i % C::STAGES], (i / C::STAGES) & 1);
        if (sh.awaited) mbar_wait_bounded(&sh.answered, sh.answers & 1);
    }
    __syncwarp();
    if (warp == 9) tmem_free(tmem, 512);
}

bool make_map(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims,
              const cuuint64_t *strides, const cuuint32_t *box) {
    auto fn = encode_fn();
    const cuuint32_t one[3] = {1, 1, 1};
    return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<void *>(base), dims,
                    strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int row_pairs(const LatentPrefillArgs &a) { return (a.max_q_len + 2 * kRows - 1) / (2 * kRows); }

template <int D, int CL>
cudaError_t launch(const LatentPrefillArgs &a, cudaStream_t stream) {
    using C = Cfg<D>;
    const cuuint64_t H = a.n_heads;
    // total_kv 0 launches no copy (every sequence with queries is flagged)
    const cuuint64_t keys = a.total_kv > 0 ? a.total_kv : 1;
    CUtensorMap mq, mkv, mr;
    const cuuint64_t dq[3] = {D + kP, H, static_cast<cuuint64_t>(a.total_q)};
    const cuuint64_t sq[2] = {(D + kP) * 2, H * (D + kP) * 2};
    const cuuint32_t bq[3] = {64, 1, kRows};
    const cuuint64_t dk[3] = {2 * D, H, keys};
    const cuuint64_t sk[2] = {2 * D * 2, H * 2 * D * 2};
    const cuuint32_t bk[3] = {64, 1, kKeys};
    const cuuint64_t dr[2] = {kP, keys};
    const cuuint64_t sr[1] = {kP * 2};
    const cuuint32_t br[2] = {64, kKeys};
    if (!make_map(&mq, a.q, 3, dq, sq, bq) || !make_map(&mkv, a.kv, 3, dk, sk, bk) ||
        !make_map(&mr, a.k_rope, 2, dr, sr, br))
        return cudaErrorNotSupported;
    auto kern = latent_prefill_kernel<D, CL>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t attr = allow_smem(kern, C::SMEM, done);
    if (attr != cudaSuccess) return attr;
    const dim3 grid(CL * row_pairs(a), a.n_heads, a.num_seqs);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = CL;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CL > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, mq, mkv, mr);
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, int sms, cudaStream_t stream) {
    // Few items: the keys of each are split over a cluster, as long as all CTAs run at
    // once (items at most: the lengths are on the device).  Resident CTAs, with 2 and
    // with 4 a cluster, in us, 128-wide heads:
    //    32 items, 512 rows behind 4000     64.4  40.3  26.9
    //    32 items, 512 rows                 14.6  13.0  12.1
    //    64 items, 2 x 512 rows behind 2000 41.7  29.3  38.4
    //   128 items, 512 rows behind 2000     44.7  58.3  78.2
    const long long items = static_cast<long long>(row_pairs(a)) * a.n_heads * a.num_seqs;
    const int cl = 4 * items <= sms ? 4 : 2 * items <= sms ? 2 : 1;
    if (a.head_dim == 128)
        return cl == 4 ? launch<128, 4>(a, stream) : cl == 2 ? launch<128, 2>(a, stream)
                                                             : launch<128, 1>(a, stream);
    return cl == 4 ? launch<64, 4>(a, stream) : cl == 2 ? launch<64, 2>(a, stream)
                                                        : launch<64, 1>(a, stream);
}

}  // namespace pkv
