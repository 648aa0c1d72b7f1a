// latent_gather.cu -- cached latent rows out of their blocks, in token order
// (paged_latent_gather): a copy, bound by memory.  A CTA takes kRows output
// rows: one thread a row finds the row's sequence (binary search over start)
// and its cache row, then all threads move 16-byte pieces, coalesced on both
// sides (a row is one contiguous piece of the cache).  72000 rows of 576 entries:
// 26.7 us, 6.2 TB/s read and written, 92 % of the copy rate (28.4 with
// the default cache policies: nothing here is used twice).
#include "pagedkv_latent.h"
#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "rope_latent.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;
constexpr int kSteps = 5;  // pieces a thread has in flight: 16 rows of 576 entries in one go

__global__ void __launch_bounds__(kThreads) latent_gather_kernel(const LatentGatherArgs a) {
    grid_dependency_wait();
    allow_dependent_launch();
    __shared__ long long src[kRows];  // cache row, or -1
    const long long first = static_cast<long long>(blockIdx.x) * kRows;
    if (threadIdx.x < kRows) {
        const long long r = first + threadIdx.x;
        long long row = -1;
        if (r < a.total && r >= a.start[0] && r < a.start[a.num_seqs]) {
            int lo = 0, hi = a.num_seqs;  // start[lo] <= r < start[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (a.start[mid] <= r) lo = mid; else hi = mid;
            }
            const long long t = r - a.start[lo];
            const long long b = t / a.block_size;
            if (t < 0 || b >= a.max_blocks_per_seq) {
                flag_error(a.err, PKV_ERRBIT_CONTEXT);
            } else {
                const int id = a.block_tables[static_cast<long long>(lo) * a.max_blocks_per_seq + b];
                if (id < 0 || id >= a.num_blocks)
                    flag_error(a.err, PKV_ERRBIT_BLOCK_ID);
                else
                    row = static_cast<long long>(id) * a.block_size + (t - b * a.block_size);
            }
        }
        src[threadIdx.x] = row;
    }
    __syncthreads();
    const int rv = a.latent_dim / 8, pv = a.rope_dim / 8, w = rv + pv;
    // i / w by the high half of a product: exact, since i * w < 2^20 < 2^32 / w
    const unsigned inv = static_cast<unsigned>((0x100000000ull + w - 1) / w);
    const uint4 *cache = static_cast<const uint4 *>(a.cache);
    uint4 *latents = static_cast<uint4 *>(a.latents), *ropes = static_cast<uint4 *>(a.ropes);
    for (int i0 = threadIdx.x; i0 < kRows * w; i0 += kSteps * kThreads) {
        uint4 x[kSteps];
        uint4 *dst[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int i = i0 + s * kThreads;
            dst[s] = nullptr;
            if (i >= kRows * w) continue;
            const int k = __umulhi(i, inv), c = i - k * w;
            if (src[k] < 0) continue;
            x[s] = __ldcs(cache + src[k] * w + c);
            dst[s] = c < rv ? latents + (first + k) * rv + c : ropes + (first + k) * pv + (c - rv);
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            if (dst[s]) __stcs(dst[s], x[s]);
    }
}

}  // namespace

cudaError_t launch_latent_gather(const LatentGatherArgs &a, cudaStream_t stream) {
    const long long blocks = (a.total + kRows - 1) / kRows;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(latent_gather_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, a);
}

}  // namespace pkv
