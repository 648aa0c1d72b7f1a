// latent_prefill.cu -- expanded latent attention of prompts
// (latent_prefill_attention): causal attention with keys [k, k_rope] of D + 64
// entries and values of D.
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

constexpr int kP = 64;          // rotated entries
constexpr int kRows = 128;      // query rows of a tile
constexpr int kKeys = 96;       // key rows of a step
constexpr int kThreads = 320;   // two softmax warpgroups, the copy warp, the MMA warp
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

struct Barriers {
    uint64_t q_full[2], s_full[2], p_ready[2][2], o_done[2], drained;
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint32_t tmem;
    int stop;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const LatentPrefillArgs a, const __grid_constant__ CUtensorMap mq,
                          const __grid_constant__ CUtensorMap mkv,
                          const __grid_constant__ CUtensorMap mr) {
    using C = Cfg<D>;
    extern __shared__ unsigned char raw[];
    __shared__ Barriers bar;
    unsigned char *base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int seq = blockIdx.z, h = blockIdx.y;
    const int pair = gridDim.x - 1 - blockIdx.x;  // the longest rows first
    grid_dependency_wait();
    allow_dependent_launch();
    const int q0 = a.q_start[seq], n = a.q_start[seq + 1] - q0;
    const int k0 = a.kv_start[seq], m = a.kv_start[seq + 1] - k0;
    if (n == 0) return;
    if (n < 0 || n > m || n > a.max_q_len || m > a.max_kv_len || q0 < 0 || k0 < 0 ||
        n > a.total_q - q0 || m > a.total_kv - k0) {
        if (threadIdx.x == 0) flag_error(a.err, PKV_ERRBIT_CONTEXT);
        return;
    }
    if (pair * 2 * kRows >= n) return;
    // key steps of the two row tiles
    int steps[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = (2 * pair + t) * kRows;
        const int last = min(first + kRows, n) - 1;
        steps[t] = first < n ? (m - n + last + kKeys) / kKeys : 0;  // ceil((m - n + last + 1) / kKeys)
    }
    const int total = max(steps[0], steps[1]);

    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bar.q_full[t], 1);
            mbar_init(&bar.s_full[t], 1);
            mbar_init(&bar.p_ready[t][0], 4);
            mbar_init(&bar.p_ready[t][1], 4);
            mbar_init(&bar.o_done[t], 1);
        }
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&bar.k_full[s], 1);
            mbar_init(&bar.k_empty[s], 1);
            mbar_init(&bar.v_full[s], 1);
            mbar_init(&bar.v_empty[s], 1);
        }
        mbar_init(&bar.drained, 1);
        bar.stop = 0;
        fence_barrier_init();
    }
    if (warp == 9) tmem_alloc(&bar.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    volatile int *stop = &bar.stop;
    // TMEM columns: S of tile t at 128 t (P in its first half), O at 256 + 128 t

    if (warp == 8) {
        if (elect_one()) {
            prefetch_tmap(&mq);
            prefetch_tmap(&mkv);
            prefetch_tmap(&mr);
            for (int t = 0; t < 2; ++t)
                if (steps[t] > 0) {
                    mbar_arrive_expect_tx(&bar.q_full[t], C::KP * kQPlane);
                    for (int p = 0; p < C::KP; ++p)
                        tma_load_3d(base + (t * C::KP + p) * kQPlane, &mq, 64 * p, h,
                                    q0 + (2 * pair + t) * kRows, &bar.q_full[t]);
                }
            int j = 0;
            for (; j < total; ++j) {
                const int s = j % C::STAGES;
                const uint32_t par = ((j / C::STAGES) & 1) ^ 1;
                unsigned char *st = base + C::Q_BYTES + s * C::STAGE_BYTES;
                const int row = k0 + j * kKeys;
                if (!wait_or_stop(&bar.k_empty[s], par, stop)) break;
                mbar_arrive_expect_tx(&bar.k_full[s], C::KP * kKPlane);
                for (int p = 0; p < D / 64; ++p)
                    tma_load_3d(st + p * kKPlane, &mkv, 64 * p, h, row, &bar.k_full[s]);
                tma_load_2d(st + (D / 64) * kKPlane, &mr, 0, row, &bar.k_full[s]);
                if (!wait_or_stop(&bar.v_empty[s], par, stop)) break;
                mbar_arrive_expect_tx(&bar.v_full[s], C::VP * kKPlane);
                for (int p = 0; p < C::VP; ++p)
                    tma_load_3d(st + (C::KP + p) * kKPlane, &mkv, D + 64 * p, h, row,
                                &bar.v_full[s]);
            }
            if (*stop) {
                // every copy in flight lands before the CTA gives its memory back
                for (int t = 0; t < 2; ++t)
                    if (steps[t] > 0) mbar_wait_bounded(&bar.q_full[t], 0);
                for (int i = max(0, j - C::STAGES + 1); i <= min(j, total - 1); ++i) {
                    mbar_wait_bounded(&bar.k_full[i % C::STAGES], (i / C::STAGES) & 1);
                    mbar_wait_bounded(&bar.v_full[i % C::STAGES], (i / C::STAGES) & 1);
                }
            }
        }
    } else if (warp == 9) {
        if (elect_one()) {
            constexpr uint32_t ds = mma_desc(kRows, kKeys, false, false);
            constexpr uint32_t dpv = mma_desc(kRows, D, false, true);
            const uint32_t q_addr = smem_addr(base), kv_addr = q_addr + C::Q_BYTES;
            auto scores = [&](int t, int j) {
                const uint32_t qa = q_addr + t * C::KP * kQPlane;
                const uint32_t ka = kv_addr + (j % C::STAGES) * C::STAGE_BYTES;
#pragma unroll
                for (int k = 0; k < 4 * C::KP; ++k)
                    mma_ss(tmem + 128 * t, smem_desc(qa + (k / 4) * kQPlane + (k % 4) * 32, 1024, 0),
                           smem_desc(ka + (k / 4) * kKPlane + (k % 4) * 32, 1024, 0), ds, k > 0);
                mma_commit(&bar.s_full[t]);
            };
            bool ok = wait_or_stop(&bar.k_full[0], 0, stop);
            for (int t = 0; t < 2 && ok; ++t)
                if (steps[t] > 0) {
                    ok = wait_or_stop(&bar.q_full[t], 0, stop);
                    if (ok) {
                        tc_fence_after();
                        scores(t, 0);
                    }
                }
            if (ok && total > C::STAGES) mma_commit(&bar.k_empty[0]);
            for (int j = 0; j < total && ok; ++j) {
                const int s = j % C::STAGES;
                const uint32_t par = (j / C::STAGES) & 1;
                const uint32_t va = kv_addr + s * C::STAGE_BYTES + C::KP * kKPlane;
                if (j + 1 < total)
                    ok = wait_or_stop(&bar.k_full[(j + 1) % C::STAGES], ((j + 1) / C::STAGES) & 1,
                                      stop);
                ok = ok && wait_or_stop(&bar.v_full[s], par, stop);
                for (int t = 0; t < 2 && ok; ++t) {
                    if (j >= steps[t]) continue;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        ok = ok && wait_or_stop(&bar.p_ready[t][half], j & 1, stop);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = half * 3; k < half * 3 + 3; ++k)
                            mma_ts(tmem + 256 + 128 * t, tmem + 128 * t + 8 * k,
                                   smem_desc(va + k * 2048, 1024, kKPlane), dpv, j > 0 || k > 0);
                    }
                    if (!ok) break;
                    if (j + 1 < steps[t])
                        scores(t, j + 1);
                    else
                        mma_commit(&bar.o_done[t]);
                }
                if (ok && j + C::STAGES < total) mma_commit(&bar.v_empty[s]);
                if (ok && j + 1 + C::STAGES < total) mma_commit(&bar.k_empty[(j + 1) % C::STAGES]);
            }
            // nothing of the tensor core is left in flight when TMEM is freed
            mma_commit(&bar.drained);
            mbar_wait_bounded(&bar.drained, 0);
        }
    } else {
        const int t = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 * (warp % 4) << 16
        const uint32_t ts = tmem + 128 * t + lanes, to = tmem + 256 + 128 * t + lanes;
        const int i = (2 * pair + t) * kRows + (threadIdx.x & 127);
        const int seen = min(m - n + i + 1, m);  // keys this row attends
        const float scale = a.scale_log2;
        float r = 0.f, l = 0.f;
        bool ok = true;
        for (int j = 0; j < steps[t]; ++j) {
            ok = warp_wait_or_stop(&bar.s_full[t], j & 1, stop);
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
            const int left = seen - j * kKeys;
            if (__any_sync(0xffffffffu, left < kKeys)) {
#pragma unroll
                for (int c = 0; c < kKeys; ++c) x[c] = c < left ? x[c] : -INFINITY;
            }
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int c = 4; c < kKeys; ++c) mx[c & 3] = fmaxf(mx[c & 3], x[c]);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
            if (j == 0) {
                r = top > -INFINITY ? top - kHead : 0.f;
            } else {
                const bool move = top - r > kHead + kLag;
                if (__any_sync(0xffffffffu, move)) {
                    // O follows the new reference; S being full, every earlier
                    // product into O is done
                    const float next = move ? top - kHead : r;
                    const float f = ex2(r - next);
                    r = next;
                    l *= f;
#pragma unroll
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(o, to + c);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(to + c, o);
                    }
                }
            }
            // values of rows beyond the sequence's keys meet weights of 0: they
            // must be finite, so the last step's are cleared
            const int valid = m - j * kKeys;
            if (valid < kKeys) {
                ok = warp_wait_or_stop(&bar.v_full[j % C::STAGES], (j / C::STAGES) & 1, stop);
                if (!ok) break;
                unsigned char *v = base + C::Q_BYTES + (j % C::STAGES) * C::STAGE_BYTES +
                                   C::KP * kKPlane;
                const int pieces = (kKeys - valid) * 8;
                for (int e = threadIdx.x & 127; e < pieces * C::VP; e += 128)
                    *reinterpret_cast<uint4 *>(v + (e / pieces) * kKPlane + valid * 128 +
                                               (e % pieces) * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t p16[16], p8[8];
#pragma unroll
                for (int c = 0; c < 24; ++c) {
                    const float y0 = ex2(fmaf(x[half * 48 + 2 * c], scale, -r));
                    const float y1 = ex2(fmaf(x[half * 48 + 2 * c + 1], scale, -r));
                    sum[(2 * c) & 3] += y0;
                    sum[(2 * c + 1) & 3] += y1;
                    if (c < 16) p16[c] = pack_half2(y0, y1); else p8[c - 16] = pack_half2(y0, y1);
                }
                tmem_st16(ts + half * 24, p16);
                tmem_st8(ts + half * 24 + 16, p8);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_ready[t][half]);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        if (ok && steps[t] > 0) ok = warp_wait_or_stop(&bar.o_done[t], 0, stop);
        if (ok && steps[t] > 0) {
            tc_fence_after();
            const float inv = 1.f / l;
            const long long row = static_cast<long long>(q0 + i) * a.n_heads + h;
            uint4 *out = reinterpret_cast<uint4 *>(static_cast<__half *>(a.out) + row * D);
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(o, to + c);
                tmem_wait_ld();
                if (i < n) {
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
            if (a.lse_out && i < n) a.lse_out[row] = (r + log2f(l)) * 0.69314718055994531f;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && bar.stop) flag_error(a.err, PKV_ERRBIT_TIMEOUT);
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

template <int D>
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
    auto kern = latent_prefill_kernel<D>;
    static std::once_flag once;
    static cudaError_t attr = cudaSuccess;
    std::call_once(once, [&] {
        attr = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (attr != cudaSuccess) return attr;
    const dim3 grid((a.max_q_len + 2 * kRows - 1) / (2 * kRows), a.n_heads, a.num_seqs);
    return launch_pdl(kern, grid, dim3(kThreads), C::SMEM, stream, a, mq, mkv, mr);
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, cudaStream_t stream) {
    return a.head_dim == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace pkv
