// kvx_cache_append: new keys and values to their slots, 16-bit values as they are, 8-bit codes rounded
// to nearest even from value * (1 / scale) in 32 bits.
//
// A thread keeps one column (plane, head, 8 elements, or 16 that become codes) and walks tokens, so shard,
// head and element offsets are computed once; only the slot changes. Reads and writes are 16 bytes a thread,
// and a CTA has as many rows of columns as make whole warps. Bound by memory: each value is read and written
// once. Measured on GB300: 8192 tokens of 8 heads of 128, both planes (67 MB) 11.7 us, 5.8 TB/s; 50001 latents
// of 576 to 8 bits (87 MB) 14.8 us, 5.9 TB/s (8-byte stores and ragged warps 17.1). With few tokens a thread
// takes one token instead of four, so that the GPU fills: 16 tokens 4.0 us, the host's time for a call.
#include "kvx_launch.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

namespace kvx {

constexpr int kAppendThreads = 512;    // at most

template <int IO> __device__ __forceinline__ float2 to_float2(uint32_t x);
template <> __device__ __forceinline__ float2 to_float2<KVX_BF16>(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 to_float2<KVX_F16>(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}

// Two codes of two values; values beyond the largest code saturate there, NaN stays.
template <int IO> __device__ __forceinline__ uint32_t codes(uint32_t x, float inverse) {
    float2 f = to_float2<IO>(x);
    f.x *= inverse;
    f.y *= inverse;
    return __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
}

// IO 0: 16-bit values copied; KVX_BF16 / KVX_F16: converted to 8 bits. UNROLL tokens per thread.
template <int IO, int UNROLL>
__global__ void __launch_bounds__(kAppendThreads) kvx_append_kernel(const __grid_constant__ AppendArgs a, int cols, int rows) {
    wait_for_earlier();
    constexpr int VEC = IO ? 16 : 8, READS = VEC / 8;             // elements of a thread
    const int my_row = threadIdx.x / cols, col = blockIdx.y * cols + threadIdx.x % cols;
    const int vecs = a.head_dim / VEC, heads = a.pool.heads_per_shard * a.pool.n_shards;
    const int plane = col / (heads * vecs), head = col / vecs % heads, vec = col % vecs;
    if (my_row >= rows || plane >= a.planes) return;
    const uint8_t *src = (plane ? a.v : a.k) + (int64_t)(head * vecs + vec) * VEC * 2;
    const int64_t stride = plane ? a.v_stride : a.k_stride;
    const int shard = head / a.pool.heads_per_shard;
    uint8_t *dst = (plane ? a.pool.v[shard] : a.pool.k[shard]) + (int64_t)(head - shard * a.pool.heads_per_shard) * a.pool.head_pitch + vec * 16;
    const float inverse = plane ? a.v_inverse : a.k_inverse;
    int64_t slot[UNROLL];
    uint4 x[UNROLL][READS];
    const int64_t t0 = (int64_t)blockIdx.x * UNROLL * rows + my_row;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int64_t t = t0 + u * rows;
        slot[u] = t < a.n_tokens ? a.slots[t] : -1;
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int64_t t = t0 + u * rows;
#pragma unroll
        for (int i = 0; i < READS; ++i)
            if (t < a.n_tokens) x[u][i] = __ldg(reinterpret_cast<const uint4 *>(src + t * stride) + i);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        if (slot[u] < 0 || slot[u] >= a.n_rows) {
            if (slot[u] != -1 && col == 0) atomicAdd(a.pool.skipped, 1ull);
            continue;
        }
        const uint32_t row = (uint32_t)slot[u], blk = row / (uint32_t)a.pool.block_size;
        uint4 *d = reinterpret_cast<uint4 *>(dst + (int64_t)blk * a.pool.block_pitch +
                                             (int64_t)(row - blk * a.pool.block_size) * a.pool.token_pitch);
        if constexpr (IO == 0) {
            *d = x[u][0];
        } else {
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                y[2 * i] = codes<IO>(x[u][i].x, inverse) | codes<IO>(x[u][i].y, inverse) << 16;
                y[2 * i + 1] = codes<IO>(x[u][i].z, inverse) | codes<IO>(x[u][i].w, inverse) << 16;
            }
            *d = make_uint4(y[0], y[1], y[2], y[3]);
        }
    }
}

template <int IO> static cudaError_t launch(const AppendArgs &a, int32_t sms, cudaStream_t stream) {
    const int64_t all = (int64_t)a.planes * a.pool.n_shards * a.pool.heads_per_shard * (a.head_dim / (IO ? 16 : 8));
    const int cols = (int)std::min<int64_t>(all, 256);
    int rows = 1;                                                  // the most threads of whole warps, up to about 256
    for (int r = 1, best = 0; r * cols <= std::max(cols, 288); ++r) {
        const int used = r * cols * 256 / ((r * cols + 31) / 32 * 32) * std::min(r * cols, 256) / 256;
        if (used >= best) best = used, rows = r;
    }
    const unsigned y = (unsigned)((all + cols - 1) / cols);
    const bool few = (a.n_tokens + rows - 1) / rows * y < 4 * sms;
    const int unroll = few ? 1 : 4, threads = (rows * cols + 31) / 32 * 32;
    const dim3 grid((unsigned)((a.n_tokens + rows * unroll - 1) / (rows * unroll)), y);
    return launch_after(few ? kvx_append_kernel<IO, 1> : kvx_append_kernel<IO, 4>, grid, threads, 0, stream, a, cols, rows);
}

cudaError_t launch_append(const AppendArgs &a, int32_t value_type, int32_t io_type, int32_t sms, cudaStream_t stream) {
    if (value_type != KVX_E4M3) return launch<0>(a, sms, stream);
    return io_type == KVX_BF16 ? launch<KVX_BF16>(a, sms, stream) : launch<KVX_F16>(a, sms, stream);
}

}  // namespace kvx
