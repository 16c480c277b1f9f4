// What the kernels over latents share: the form of a partial result, and what they leave for the joining kernel.
#pragma once

#include "kvx_attend.cuh"
#include "kvx_waits.cuh"

namespace kvx {

constexpr int kLatentHeads = 16;                                                       // query heads at a time
constexpr int kLatentFloat4 = kLatentHeads * kCacheMaxLatentValue / 4;                 // of a partial result
constexpr int kLatentPartial = kLatentFloat4 * 16 + 2 * kLatentHeads * 4;              // O, m, l

// Place of value element d of query head h in a partial result: float4s as kvx_latent.cu's lanes hold them.
__device__ __forceinline__ int partial_at(int d, int h) {
    return ((((d >> 6) * 2 + (h >> 3)) * 2 + (h & 1)) * 2 + (d >> 2 & 1)) * 128 + ((d >> 3 & 7) * 4 + (h >> 1 & 3)) * 4 + (d & 3);
}

// What a CTA leaves for the joining kernel: the segment that begins in its stretch and goes on after it (pieces 0: none).
struct OpenSegment {
    int32_t r, seg, pieces, cta;       // cta: of the first piece, for the joining kernel alone
};

cudaError_t launch_latent_join(const AttendArgs &a, int32_t io, int ctas, int32_t sms, cudaStream_t stream);       // kvx_latent.cu
cudaError_t launch_latent_tensor(const AttendArgs &a, int32_t vt, int32_t io, int32_t sms, cudaStream_t stream);   // kvx_latent_tensor.cu

}  // namespace kvx
