// kvx_cache_attend over one plane of latents, of which the leading elements are the value.
#include "kvx_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

namespace kvx {

template <int T> __device__ __forceinline__ float value_at(const uint8_t *p, int i);
template <> __device__ __forceinline__ float value_at<KVX_BF16>(const uint8_t *p, int i) {
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
}
template <> __device__ __forceinline__ float value_at<KVX_F16>(const uint8_t *p, int i) {
    return __half2float(reinterpret_cast<const __half *>(p)[i]);
}
template <> __device__ __forceinline__ float value_at<KVX_E4M3>(const uint8_t *p, int i) {
    return (float)reinterpret_cast<const __nv_fp8_e4m3 *>(p)[i];
}

template <int T> __device__ __forceinline__ void put(uint8_t *p, int i, float x);
template <> __device__ __forceinline__ void put<KVX_BF16>(uint8_t *p, int i, float x) {
    reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
}
template <> __device__ __forceinline__ void put<KVX_F16>(uint8_t *p, int i, float x) {
    reinterpret_cast<__half *>(p)[i] = __float2half_rn(x);
}

constexpr int kWarps = 8;
constexpr int kPer = (kCacheMaxLatent + 31) / 32;

// One CTA per (query head, request); a warp takes every kWarps-th position with an online softmax, and
// the warps' sums are joined in shared memory.
template <int VT, int IO>
__global__ void __launch_bounds__(32 * kWarps) kvx_attend_latent(const __grid_constant__ AttendArgs a) {
    __shared__ float s_max[kWarps], s_sum[kWarps], s_out[kWarps][kCacheMaxLatentValue];
    const int head = blockIdx.x, r = blockIdx.y + blockIdx.z * 65535;
    if (r >= a.n_reqs) return;
    const int kvh = head / (a.n_q_heads / a.n_kv_heads), shard = kvh / a.pool.heads_per_shard;
    const int64_t head_off = (int64_t)(kvh - shard * a.pool.heads_per_shard) * a.pool.head_pitch;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t cap = (int64_t)a.max_blocks * a.pool.block_size;
    int64_t len = a.seq_len[r];
    if ((len < 0 || len > cap) && head == 0 && threadIdx.x == 0) atomicAdd(a.pool.skipped, 1ull);
    len = max((int64_t)0, min(len, cap));
    const int64_t first = a.window ? max((int64_t)0, len - a.window) : 0;
    float q[kPer], acc[kPer] = {};
    const uint8_t *qp = a.q + r * a.q_stride + (int64_t)head * a.head_dim * 2;
#pragma unroll
    for (int i = 0; i < kPer; ++i) q[i] = lane + 32 * i < a.head_dim ? value_at<IO>(qp, lane + 32 * i) * a.scale : 0.0f;
    float top = -INFINITY, sum = 0.0f;
    for (int64_t t = first + w; t < len; t += kWarps) {
        const int64_t col = t / a.pool.block_size;
        const int32_t blk = a.block_table[r * a.table_stride + col];
        if (blk < 0 || blk >= a.pool.n_blocks) {
            if (lane == 0 && head == 0) atomicAdd(a.pool.skipped, 1ull);
            continue;
        }
        const int64_t off = blk * a.pool.block_pitch + (t - col * a.pool.block_size) * a.pool.token_pitch + head_off;
        const uint8_t *k = a.pool.k[shard] + off, *v = a.pool.v[shard] + off;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < a.head_dim) s += q[i] * value_at<VT>(k, lane + 32 * i);
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        const float m = fmaxf(top, s), old = top == m ? 1.0f : exp2f(top - m), p = exp2f(s - (m == -INFINITY ? 0.0f : m));
        top = m;
        sum = sum * old + p;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < a.v_dim) acc[i] = acc[i] * old + p * value_at<VT>(v, lane + 32 * i);
    }
    if (lane == 0) {
        s_max[w] = top;
        s_sum[w] = sum;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (lane + 32 * i < a.v_dim) s_out[w][lane + 32 * i] = acc[i];
    __syncthreads();
    float m = -INFINITY, l = 0.0f;
    for (int i = 0; i < kWarps; ++i) m = fmaxf(m, s_max[i]);
    for (int i = 0; i < kWarps; ++i) l += s_max[i] == -INFINITY ? s_sum[i] : s_sum[i] * exp2f(s_max[i] - m);
    for (int d = threadIdx.x; d < a.v_dim; d += blockDim.x) {
        float o = 0.0f;
        for (int i = 0; i < kWarps; ++i) o += s_max[i] == -INFINITY ? s_out[i][d] : s_out[i][d] * exp2f(s_max[i] - m);
        put<IO>(a.out + r * a.out_stride + (int64_t)head * a.v_dim * 2, d, l == 0.0f ? 0.0f : o / l * a.v_scale);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[(int64_t)r * a.n_q_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

cudaError_t launch_attend_latent(const AttendArgs &a, int32_t vt, int32_t io, int32_t, cudaStream_t stream) {
    const dim3 grid(a.n_q_heads, std::min(a.n_reqs, 65535), (a.n_reqs + 65534) / 65535);
    if (vt == KVX_BF16) kvx_attend_latent<KVX_BF16, KVX_BF16><<<grid, 32 * kWarps, 0, stream>>>(a);
    else if (vt == KVX_F16) kvx_attend_latent<KVX_F16, KVX_F16><<<grid, 32 * kWarps, 0, stream>>>(a);
    else if (io == KVX_BF16) kvx_attend_latent<KVX_E4M3, KVX_BF16><<<grid, 32 * kWarps, 0, stream>>>(a);
    else kvx_attend_latent<KVX_E4M3, KVX_F16><<<grid, 32 * kWarps, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}

}  // namespace kvx
