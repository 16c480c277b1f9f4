// kvx_cache_attend_shared over planes of KVX_F16, queries and outputs in KVX_F16: the positions behind the prefixes.
#include "kvx_attend_planes.cuh"

namespace kvx {

cudaError_t launch_rest_f16(const SharedArgs &s, int32_t sms, cudaStream_t stream) {
    return launch_rest_planes<KVX_F16, KVX_F16>(s, sms, stream);
}

}  // namespace kvx
