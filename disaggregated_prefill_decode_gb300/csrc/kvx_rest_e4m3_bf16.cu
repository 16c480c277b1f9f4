// kvx_cache_attend_shared over planes of KVX_E4M3, queries and outputs in KVX_BF16: the positions behind the prefixes.
#include "kvx_attend_planes.cuh"

namespace kvx {

cudaError_t launch_rest_e4m3_bf16(const SharedArgs &s, int32_t sms, cudaStream_t stream) {
    return launch_rest_planes<KVX_E4M3, KVX_BF16>(s, sms, stream);
}

}  // namespace kvx
