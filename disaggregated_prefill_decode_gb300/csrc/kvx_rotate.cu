// kvx_cache_append_rotated: queries and keys normed over each head and turned by their token's position, the queries to an array,
// the keys, and the values as they are, to their slots; everything between the read and the one rounding in 32 bits.
//
// A pair (a, b) of a head at position p becomes m (a cos - b sin, b cos + a sin) of p times the pair's frequency. The angle is
// taken in turns, as a 64-bit fraction: position times frequency modulo 2^64 is the fraction of a turn that counts, exactly,
// however far the position is (in 32 bits it would be off by 2^-24 of the angle: 0.1 radians at 10^6). Its upper 32 bits go to sincospif.
//
// A warp takes one token and some of its heads, 32 / LANES of them at a time. A lane has two vectors of 8 elements of a head
// (or twice two): with halves, the two that turn with one another, so no element changes lanes; sines and cosines are computed once for all
// heads. Bound by memory: each value is read and written once, in 16 bytes a lane.
#include "kvx_attend.cuh"

#include <cuda_fp8.h>

#include <algorithm>

namespace kvx {

constexpr int kRotateThreads = 256, kRotateWarps = kRotateThreads / 32;

// A lane's two vectors of a head, and what becomes of them.
struct RotateVecs {
    int a, b;                          // -1: none
    bool turns_a, turns_b;             // halves: both or none
    bool norm_a, norm_b;
};

// Slot s of a head: the vectors that turn with one another, or two neighbours in a list of what is left.
__device__ __forceinline__ RotateVecs rotate_vecs(const RotateArgs &r, int s) {
    const int vecs = r.head_dim / 8, begin = r.begin / 8, turned = r.turned / 8;
    RotateVecs v = {-1, -1, false, false, false, false};
    if (!r.pairs && turned) {
        const int couples = turned / 2, rest = vecs - turned, t = s - couples, half = (rest + 1) / 2;
        if (s < couples) {
            v.a = begin + s;
            v.b = v.a + couples;
            v.turns_a = v.turns_b = true;
        } else {
            if (t < half) v.a = t < begin ? t : t + turned;
            if (t < half && t + half < rest) v.b = t + half < begin ? t + half : t + half + turned;
        }
    } else {
        const int half = (vecs + 1) / 2;
        if (s < half) v.a = s;
        if (s < half && s + half < vecs) v.b = s + half;
        v.turns_a = v.a >= begin && v.a < begin + turned;
        v.turns_b = v.b >= begin && v.b < begin + turned;
    }
    v.norm_a = v.a >= 0 && v.a * 8 < r.norm_dim;
    v.norm_b = v.b >= 0 && v.b * 8 < r.norm_dim;
    return v;
}

template <int IO> __device__ __forceinline__ void widen(const uint4 &x, float (&y)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack<IO>(w[i]);
        y[2 * i] = f.x;
        y[2 * i + 1] = f.y;
    }
}

template <int IO> __device__ __forceinline__ uint4 narrow(const float (&y)[8]) {
    return make_uint4(pack<IO>(y[0], y[1]), pack<IO>(y[2], y[3]), pack<IO>(y[4], y[5]), pack<IO>(y[6], y[7]));
}

// Codes of eight values; those beyond the largest saturate there, NaN stays.
__device__ __forceinline__ uint2 codes(const float (&y)[8], float inverse) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i] * inverse, y[2 * i + 1] * inverse), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

template <int IO, bool F8, int LANES, int NP>
__global__ void __launch_bounds__(kRotateThreads) kvx_rotate_kernel(const __grid_constant__ RotateArgs r) {
    constexpr int AT_ONCE = 32 / LANES, AHEAD = NP == 1 ? 4 : 1;      // heads of a warp; rounds whose reads are under way together
    wait_for_earlier();
    const int lane = threadIdx.x & 31, in_head = lane % LANES, which = lane / LANES;
    const int64_t item = (int64_t)blockIdx.x * kRotateWarps + (threadIdx.x >> 5);
    const int64_t token = item / r.parts;
    const int part = (int)(item - token * r.parts);
    if (token >= r.n_tokens) return;
    const int64_t slot = r.slots[token];
    if (slot < 0 || slot >= r.n_rows) {
        if (slot != -1 && part == 0 && lane == 0) atomicAdd(r.pool.skipped, 1ull);
        return;
    }
    RotateVecs v[NP];
    float cosine[NP][8], sine[NP][8];
    const int64_t pos = r.turned ? r.positions[token] : 0;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const int s = in_head + LANES * n;
        v[n] = rotate_vecs(r, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // halves: pair 8 s + i of element i of both vectors; pairs: four of each vector
            const int at = !r.pairs ? 8 * s + i : i < 4 ? (v[n].a - r.begin / 8) * 4 + i : (v[n].b - r.begin / 8) * 4 + i - 4;
            cosine[n][i] = 1.0f;
            sine[n][i] = 0.0f;
            if (i < 4 || !r.pairs ? v[n].turns_a : v[n].turns_b) {
                const int32_t turn = (int32_t)((r.turns[at] * (uint64_t)pos) >> 32);
                sincospif((float)turn * 0x1p-31f, &sine[n][i], &cosine[n][i]);
                sine[n][i] *= r.magnitude;
                cosine[n][i] *= r.magnitude;
            }
        }
    }
    const uint32_t row = (uint32_t)slot, blk = row / (uint32_t)r.pool.block_size;
    const int64_t at_slot = (int64_t)blk * r.pool.block_pitch + (int64_t)(row - blk * r.pool.block_size) * r.pool.token_pitch;
    const int heads = r.n_q_heads + r.planes * r.n_kv_heads;          // queries, keys, values
    const int begin = (int)((int64_t)heads * part / r.parts), end = (int)((int64_t)heads * (part + 1) / r.parts);
    const int row_bytes = r.head_dim * 2;
    for (int h0 = begin; h0 < end; h0 += AT_ONCE * AHEAD) {
        uint4 x[AHEAD][NP][2];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int h = h0 + u * AT_ONCE + which;
            if (h >= end) continue;
            const int kv = h - r.n_q_heads;
            const uint8_t *src = kv < 0 ? r.q + token * r.q_stride + (int64_t)h * row_bytes
                                 : kv < r.n_kv_heads ? r.k + token * r.k_stride + (int64_t)kv * row_bytes
                                                     : r.v + token * r.v_stride + (int64_t)(kv - r.n_kv_heads) * row_bytes;
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                x[u][n][0] = v[n].a >= 0 ? __ldcs(reinterpret_cast<const uint4 *>(src) + v[n].a) : make_uint4(0, 0, 0, 0);
                x[u][n][1] = v[n].b >= 0 ? __ldcs(reinterpret_cast<const uint4 *>(src) + v[n].b) : make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (h0 + u * AT_ONCE >= end) break;                       // the whole warp
            const int h = h0 + u * AT_ONCE + which, kv = h - r.n_q_heads;
            const bool in = h < end, value = kv >= r.n_kv_heads;
            const uint8_t *weight = value ? nullptr : kv < 0 ? r.q_weight : r.k_weight;
            float y[NP][2][8];
            float sum = 0.0f;
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                if (!in) x[u][n][0] = x[u][n][1] = make_uint4(0, 0, 0, 0);
                widen<IO>(x[u][n][0], y[n][0]);
                widen<IO>(x[u][n][1], y[n][1]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (v[n].norm_a) sum = fmaf(y[n][0][i], y[n][0][i], sum);
                    if (v[n].norm_b) sum = fmaf(y[n][1][i], y[n][1][i], sum);
                }
            }
            if (r.q_weight || r.k_weight) {                           // of the whole warp: some lanes may have other heads
#pragma unroll
                for (int d = 1; d < LANES; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
            }
            if (weight && in) {
                const float inverse = rsqrtf(sum * r.norm_inverse + r.eps);
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    float w[8];
                    if (v[n].norm_a) {
                        widen<IO>(__ldg(reinterpret_cast<const uint4 *>(weight) + v[n].a), w);
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[n][0][i] *= inverse * w[i];
                    }
                    if (v[n].norm_b) {
                        widen<IO>(__ldg(reinterpret_cast<const uint4 *>(weight) + v[n].b), w);
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[n][1][i] *= inverse * w[i];
                    }
                }
            }
            if (!in) continue;
            if (!value)
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    if (!r.pairs) {
                        if (v[n].turns_a)
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float a = y[n][0][i], b = y[n][1][i];
                                y[n][0][i] = a * cosine[n][i] - b * sine[n][i];
                                y[n][1][i] = b * cosine[n][i] + a * sine[n][i];
                            }
                    } else {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            if (k ? v[n].turns_b : v[n].turns_a)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float a = y[n][k][2 * i], b = y[n][k][2 * i + 1];
                                    y[n][k][2 * i] = a * cosine[n][4 * k + i] - b * sine[n][4 * k + i];
                                    y[n][k][2 * i + 1] = b * cosine[n][4 * k + i] + a * sine[n][4 * k + i];
                                }
                    }
                }
            if (kv < 0) {
                uint4 *dst = reinterpret_cast<uint4 *>(r.q_out + token * r.out_stride + (int64_t)h * row_bytes);
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    if (v[n].a >= 0) dst[v[n].a] = narrow<IO>(y[n][0]);
                    if (v[n].b >= 0) dst[v[n].b] = narrow<IO>(y[n][1]);
                }
            } else {
                const int head = value ? kv - r.n_kv_heads : kv, shard = head / r.pool.heads_per_shard;
                uint8_t *dst = (value ? r.pool.v[shard] : r.pool.k[shard]) + (int64_t)(head - shard * r.pool.heads_per_shard) * r.pool.head_pitch + at_slot;
                const float inverse = value ? r.v_inverse : r.k_inverse;
#pragma unroll
                for (int n = 0; n < NP; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int vec = k ? v[n].b : v[n].a;
                        if (vec < 0) continue;
                        if constexpr (F8) reinterpret_cast<uint2 *>(dst)[vec] = codes(y[n][k], inverse);
                        else reinterpret_cast<uint4 *>(dst)[vec] = narrow<IO>(y[n][k]);
                    }
            }
        }
    }
}

template <int IO, bool F8, int LANES, int NP> static cudaError_t launch(RotateArgs a, int32_t sms, cudaStream_t stream) {
    // A token's heads go to as many warps as fill the GPU: each of them computes the token's sines and cosines again.
    const int64_t rounds = (a.n_q_heads + a.planes * a.n_kv_heads + 32 / LANES - 1) / (32 / LANES);
    a.parts = (int32_t)std::min<int64_t>(rounds, std::max<int64_t>(1, (32 * sms + a.n_tokens - 1) / a.n_tokens));
    const int64_t ctas = (a.n_tokens * a.parts + kRotateWarps - 1) / kRotateWarps;
    return launch_after(kvx_rotate_kernel<IO, F8, LANES, NP>, dim3((unsigned)ctas), kRotateThreads, 0, stream, a);
}

template <int IO, bool F8> static cudaError_t launch_dim(const RotateArgs &a, int32_t sms, cudaStream_t stream) {
    // Slots of a head: each holds two vectors, and both lists of them may end in half of one.
    const int vecs = a.head_dim / 8, slots = a.turned && !a.pairs ? a.turned / 16 + (vecs - a.turned / 8 + 1) / 2 : (vecs + 1) / 2;
    if (slots <= 4) return launch<IO, F8, 4, 1>(a, sms, stream);
    if (slots <= 8) return launch<IO, F8, 8, 1>(a, sms, stream);
    if (slots <= 16) return launch<IO, F8, 16, 1>(a, sms, stream);
    return launch<IO, F8, 32, 2>(a, sms, stream);
}

cudaError_t launch_rotate(const RotateArgs &a, int32_t value_type, int32_t io_type, int32_t sms, cudaStream_t stream) {
    if (value_type == KVX_E4M3)
        return io_type == KVX_BF16 ? launch_dim<KVX_BF16, true>(a, sms, stream) : launch_dim<KVX_F16, true>(a, sms, stream);
    return io_type == KVX_BF16 ? launch_dim<KVX_BF16, false>(a, sms, stream) : launch_dim<KVX_F16, false>(a, sms, stream);
}

}  // namespace kvx
