// kvx_cache_attend's launcher. The kernels: kvx_attend_planes.cuh, kvx_latent.cu.
#include "kvx_internal.h"

namespace kvx {

// Counters of the segments that cross CTAs, then partial results: two per CTA and one per warp (kvx_attend_planes.cuh).
size_t attend_scratch_bytes(int32_t sms, bool latent) {
    if (latent) return latent_scratch_bytes(sms);
    return kScratchCounters * sizeof(uint32_t) + (size_t)sms * kScratchPerSm;
}

cudaError_t launch_attend(const AttendArgs &a, int32_t vt, int32_t io, int32_t sms, cudaStream_t stream) {
    if (a.latent) return launch_attend_latent(a, vt, io, sms, stream);
    if (vt == KVX_BF16) return launch_attend_bf16(a, sms, stream);
    if (vt == KVX_F16) return launch_attend_f16(a, sms, stream);
    return io == KVX_BF16 ? launch_attend_e4m3_bf16(a, sms, stream) : launch_attend_e4m3_f16(a, sms, stream);
}

}  // namespace kvx
