// kvx_cache_attend_shared over planes of KVX_F16, queries and outputs in KVX_F16: the prefixes.
#include "kvx_shared.cuh"

namespace kvx {

cudaError_t launch_shared_f16(const SharedArgs &s, int32_t sms, cudaStream_t stream) {
    return launch_shared_type<KVX_F16, KVX_F16>(s, sms, stream);
}

}  // namespace kvx
