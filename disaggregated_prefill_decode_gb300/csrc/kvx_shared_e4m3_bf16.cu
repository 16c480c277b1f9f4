// kvx_cache_attend_shared over planes of KVX_E4M3, queries and outputs in KVX_BF16: the prefixes.
#include "kvx_shared.cuh"

namespace kvx {

cudaError_t launch_shared_e4m3_bf16(const SharedArgs &s, int32_t sms, cudaStream_t stream) {
    return launch_shared_type<KVX_E4M3, KVX_BF16>(s, sms, stream);
}

}  // namespace kvx
