// kvx_cache_attend over planes of KVX_E4M3, queries and outputs in KVX_BF16.
#include "kvx_attend_planes.cuh"

namespace kvx {

cudaError_t launch_attend_e4m3_bf16(const AttendArgs &a, int32_t sms, cudaStream_t stream) {
    return launch_planes<KVX_E4M3, KVX_BF16>(a, sms, stream);
}

}  // namespace kvx
