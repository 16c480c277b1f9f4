// kvx_cache_append_rotated: queries and keys normed over each head and turned by their token's position, the queries to an array,
// the keys, and the values as they are, to their slots; everything between the read and the one rounding in 32 bits.
//
// A pair (a, b) of a head at position p becomes m (a cos - b sin, b cos + a sin) of p times the pair's frequency. The angle is
// taken in turns, as a 64-bit fraction: position times frequency modulo 2^64 is the fraction of a turn that counts, exactly,
// however far the position is (in 32 bits it would be off by 2^-24 of the angle: 0.06 radians at 10^6). Its upper 32 bits go to
// sincospif, as a float: 2^-26 of a turn. The frequency's own 53 bits are off by 2^-55 of a turn a position.
//
// A warp takes a token (or a part of its heads), then another one, 32 / LANES heads a round. A lane has two vectors of 8 elements of a head
// (or twice two): with halves, the two that turn with one another, so no element changes lanes; sines, cosines and their products
// with the weights are computed once for all heads. Bound by memory: each value is read and written once, in 16 bytes a lane, and what counts
// is bytes on their way: asynchronous copies of four rounds into places of shared memory that the lane itself reads back.
//
// Measured on GB300: 8192 tokens of 64 + 8 + 8 heads of 128 (336 MB) 54.7 us, 6.1 TB/s; 64 latents with 16 query heads 5.3, the host's time for a
// call, 1158 of them 14.4, 5000 with 24 heads 70 (4.1 TB/s). Steps: a warp a token, reads of four heads ahead in registers 86.7 us; a persistent warp, sines by the warp 68; no exceptions for
// lanes where whole heads turn (31 million instructions, 42) 70; the next rounds' reads over tokens, in registers 74; in shared memory
// 63 with 24 warps an SM, 58 with 16 (8 rounds ahead 71 and 59: the more rows at once, the slower the memory); tokens in two parts 55.
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

// Slot s of a head: the vectors that turn with one another, or two neighbours in a list of what is left. With two slots a lane (NP) those
// of the first ones are 64 vectors in a row, so that what turns of a latent is in the second ones alone.
template <int NP> __device__ __forceinline__ RotateVecs rotate_vecs(const RotateArgs &r, int s) {
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
        const int half = (vecs + 1) / 2, a = NP == 1 ? s : s / 32 * 64 + s % 32, b = NP == 1 ? s + half : a + 32;
        if (NP == 1 ? s < half : a < vecs) v.a = a;
        if (v.a >= 0 && b < vecs) v.b = b;
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

enum { kQueries, kKeys, kValues };

// A warp's rounds: 32 / LANES heads of one kind a round, read AHEAD rounds before, over tokens too; a lane's two vectors (or twice two)
// of one. WHOLE: every element of a head turns, and all of them are normed or none; no lane then has an exception.
template <int IO, bool F8, int LANES, int NP, bool PAIRS, bool WHOLE> struct Rotate {
    static constexpr int AT_ONCE = 32 / LANES;                        // heads of a round
    static constexpr int AHEAD = 4;                                // rounds whose reads are under way
    static constexpr int RING = AHEAD * NP * 1024;                    // bytes of a warp's ring
    using Vectors = uint4[NP][2];
    const RotateArgs &r;
    float2 *const turned;              // of the warp, in shared memory: sine and cosine of each pair at the token's position
    RotateVecs v[NP];
    int slot_of[NP];
    bool some[NP];                     // whether any lane has something that turns
    int64_t token, at_slot;
    // The weights of a kind of heads, and what they make of the sines and cosines: (a, b) becomes (a by[0] - b by[3], b by[2] + a by[1]).
    float by[NP][4][8];

    __device__ __forceinline__ Rotate(const RotateArgs &args, float2 *shared) : r(args), turned(shared) {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            slot_of[n] = threadIdx.x % LANES + LANES * n;
            v[n] = rotate_vecs<NP>(r, slot_of[n]);
            some[n] = WHOLE || __any_sync(~0u, v[n].turns_a || v[n].turns_b);
        }
    }

    // To a token: each lane has some of the pairs.
    __device__ __forceinline__ void go(int64_t t, int64_t slot, int64_t pos) {
        token = t;
        __syncwarp();
        for (int p = threadIdx.x & 31; p < r.turned / 2; p += 32) {
            const int32_t turn = (int32_t)((r.turns[p] * (uint64_t)pos) >> 32);
            float2 y;
            sincospif((float)turn * 0x1p-31f, &y.x, &y.y);
            turned[p] = make_float2(y.x * r.magnitude, y.y * r.magnitude);
        }
        __syncwarp();
        const uint32_t row = (uint32_t)slot, blk = row / (uint32_t)r.pool.block_size;
        at_slot = (int64_t)blk * r.pool.block_pitch + (int64_t)(row - blk * r.pool.block_size) * r.pool.token_pitch;
    }

    __device__ __forceinline__ static int which() { return (threadIdx.x & 31) / LANES; }

    __device__ __forceinline__ void weigh(const uint8_t *weight) {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            if (!F8 && !weight && !some[n]) continue;              // copied as they are
            float f[2][8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (weight && (WHOLE || (k ? v[n].norm_b : v[n].norm_a))) widen<IO>(__ldg(reinterpret_cast<const uint4 *>(weight) + (k ? v[n].b : v[n].a)), f[k]);
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[k][i] = 1.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {                          // pair i: elements i of both vectors, or 2i and 2i + 1 of all sixteen
                const float wa = !PAIRS ? f[0][i] : f[i / 4][i % 4 * 2], wb = !PAIRS ? f[1][i] : f[i / 4][i % 4 * 2 + 1];
                const int at = !PAIRS ? 8 * slot_of[n] + i : i < 4 ? (v[n].a - r.begin / 8) * 4 + i : (v[n].b - r.begin / 8) * 4 + i - 4;
                const float2 y = WHOLE || (i < 4 || !PAIRS ? v[n].turns_a : v[n].turns_b) ? turned[at] : make_float2(0.0f, 1.0f);
                by[n][0][i] = wa * y.y;
                by[n][1][i] = wa * y.x;
                by[n][2][i] = wb * y.y;
                by[n][3][i] = wb * y.x;
            }
        }
    }

    // What this lane has of round `at` of a kind's heads: into its places of a stage of the ring, which it alone reads back.
    __device__ __forceinline__ void read(uint32_t stage, const uint8_t *src, int at, int heads) const {
        const int h = at * AT_ONCE + which();
        const uint8_t *const p = src + (h < heads ? h : 0) * (r.head_dim * 2);
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            if (WHOLE || v[n].a >= 0) copy_async(stage + n * 1024, p + v[n].a * 16, h < heads);
            if (WHOLE || v[n].b >= 0) copy_async(stage + n * 1024 + 512, p + v[n].b * 16, h < heads);
        }
    }
    __device__ __forceinline__ static void read_back(Vectors &y, uint32_t stage) {
#pragma unroll
        for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t z[4];
                shared_read(z, stage + n * 1024 + k * 512);
                y[n][k] = make_uint4(z[0], z[1], z[2], z[3]);
            }
    }

    template <int KIND> __device__ __forceinline__ void round(const Vectors &x, int at) const {
        const int heads = KIND == kQueries ? r.n_q_heads : r.n_kv_heads;
        const uint8_t *const weight = KIND == kQueries ? r.q_weight : KIND == kKeys ? r.k_weight : nullptr;
        const int h = at * AT_ONCE + which();
        constexpr bool NARROWS = F8 && KIND != kQueries;
        float y[NP][2][8];
        bool as_is[NP];
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            as_is[n] = !NARROWS && (KIND == kValues || (!weight && !some[n]));
            if (as_is[n]) continue;
            widen<IO>(x[n][0], y[n][0]);
            widen<IO>(x[n][1], y[n][1]);
        }
        float inverse = 1.0f;
        if (weight) {
            float sum = 0.0f;
#pragma unroll
            for (int n = 0; n < NP; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float even = 0.0f, odd = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        even = fmaf(y[n][k][i], y[n][k][i], even);
                        odd = fmaf(y[n][k][i + 1], y[n][k][i + 1], odd);
                    }
                    sum += WHOLE || (k ? v[n].norm_b : v[n].norm_a) ? even + odd : 0.0f;
                }
#pragma unroll
            for (int d = 1; d < LANES; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
            inverse = rsqrtf(fmaf(sum, r.norm_inverse, r.eps));
        }
        if (h >= heads) return;
        uint8_t *dst = r.q_out + token * r.out_stride + h * (r.head_dim * 2);
        if constexpr (KIND != kQueries) {
            const int shard = h / r.pool.heads_per_shard;
            dst = (KIND == kKeys ? r.pool.k[shard] : r.pool.v[shard]) + (int64_t)(h - shard * r.pool.heads_per_shard) * r.pool.head_pitch + at_slot;
        }
        auto put = [&](int vec, const float (&z)[8]) {
            if (!WHOLE && vec < 0) return;
            if constexpr (F8 && KIND != kQueries) reinterpret_cast<uint2 *>(dst)[vec] = codes(z, KIND == kKeys ? r.k_inverse : r.v_inverse);
            else reinterpret_cast<uint4 *>(dst)[vec] = narrow<IO>(z);
        };
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            if (as_is[n]) {
                if (WHOLE || v[n].a >= 0) reinterpret_cast<uint4 *>(dst)[v[n].a] = x[n][0];
                if (WHOLE || v[n].b >= 0) reinterpret_cast<uint4 *>(dst)[v[n].b] = x[n][1];
                continue;
            }
            if constexpr (KIND != kValues) {
                const float of_a = WHOLE || v[n].norm_a ? inverse : 1.0f, of_b = WHOLE || v[n].norm_b ? inverse : 1.0f;
#pragma unroll
                for (int k = 0; k < 2; ++k) {                      // halves: both vectors at once, in the first turn
                    if (!PAIRS && k) break;
                    const bool turns = WHOLE || (k ? v[n].turns_b : v[n].turns_a);
#pragma unroll
                    for (int i = 0; i < (PAIRS ? 4 : 8); ++i) {
                        float &a = PAIRS ? y[n][k][2 * i] : y[n][0][i], &b = PAIRS ? y[n][k][2 * i + 1] : y[n][1][i];
                        const int j = PAIRS ? 4 * k + i : i;
                        const float sa = a * (PAIRS && k ? of_b : of_a), sb = b * (PAIRS && !k ? of_a : of_b);
                        a = turns ? sa * by[n][0][j] - sb * by[n][3][j] : sa * by[n][0][j];
                        b = turns ? sb * by[n][2][j] + sa * by[n][1][j] : sb * by[n][2][j];
                    }
                }
            }
            put(v[n].a, y[n][0]);
            put(v[n].b, y[n][1]);
        }
    }
};

template <int IO, bool F8, int LANES, int NP, bool PAIRS, bool WHOLE>
__global__ void __launch_bounds__(kRotateThreads, NP == 1 ? 2 : 1) kvx_rotate_kernel(const __grid_constant__ RotateArgs r) {
    using Warp = Rotate<IO, F8, LANES, NP, PAIRS, WHOLE>;
    __shared__ float2 s_turned[kRotateWarps][kRotateMaxPairs];
    extern __shared__ __align__(16) uint8_t s_ring[];
    wait_for_earlier();
    Warp warp(r, s_turned[threadIdx.x >> 5]);
    const int q_rounds = (r.n_q_heads + Warp::AT_ONCE - 1) / Warp::AT_ONCE, kv_rounds = (r.n_kv_heads + Warp::AT_ONCE - 1) / Warp::AT_ONCE;
    const int keys = q_rounds, values = q_rounds + kv_rounds, all = q_rounds + r.planes * kv_rounds;       // first rounds
    // A warp has rounds [from, upto) of every so-manyth token, or (line) an equal stretch of one line of all tokens' rounds.
    int from = (int)((uint32_t)all * blockIdx.y / gridDim.y), upto = (int)((uint32_t)all * (blockIdx.y + 1) / gridDim.y);
    int64_t step = (int64_t)gridDim.x * kRotateWarps, token = (int64_t)blockIdx.x * kRotateWarps + (threadIdx.x >> 5);
    int64_t left = token < r.n_tokens ? (int64_t)((uint32_t)(r.n_tokens - 1 - token) / (uint32_t)step + 1) * (upto - from) : 0;
    int at = from;
    if (NP > 1 && r.line) {
        const int64_t begin = r.n_tokens * all * token / step;
        left = r.n_tokens * all * (token + 1) / step - begin;
        token = begin / all;
        at = (int)(begin - token * all);
        step = 1;
    }
    int64_t far = token, far_left = left, slot = -1, pos = 0;
    int far_at = at;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(s_ring) + (threadIdx.x >> 5) * Warp::RING + (threadIdx.x & 31) * 16;
    auto read = [&](int stage) {                                      // the next round to be read
        if (far_left > 0) {
            const uint32_t to = ring + stage * (NP * 1024);
            if (far_at < keys) warp.read(to, r.q + far * r.q_stride, far_at, r.n_q_heads);
            else if (far_at < values) warp.read(to, r.k + far * r.k_stride, far_at - keys, r.n_kv_heads);
            else warp.read(to, r.v + far * r.v_stride, far_at - values, r.n_kv_heads);
            --far_left;
            if (++far_at == upto) {
                far_at = from;
                far += step;
            }
        }
        copies_commit();
    };
    auto look_up = [&](int64_t t) {
        slot = t < r.n_tokens ? r.slots[t] : -1;
        pos = t < r.n_tokens && r.turned ? r.positions[t] : 0;
    };
    look_up(token);
    for (int u = 0; u < Warp::AHEAD - 1; ++u) read(u);
    bool live = false, fresh = true;
    for (int stage = 0; left > 0; --left, stage = stage + 1 == Warp::AHEAD ? 0 : stage + 1) {
        read(stage ? stage - 1 : Warp::AHEAD - 1);
        if (fresh) {
            const int64_t here = slot;
            live = here >= 0 && here < r.n_rows;
            if (live) warp.go(token, here, pos);
            else if (here != -1 && at == 0 && (threadIdx.x & 31) == 0) atomicAdd(r.pool.skipped, 1ull);
            look_up(token + step);
        }
        copies_wait<Warp::AHEAD - 1>();
        if (live) {
            if ((fresh && at < values) || at == keys) warp.weigh(at < keys ? r.q_weight : r.k_weight);
            typename Warp::Vectors x;
            Warp::read_back(x, ring + stage * (NP * 1024));
            if (at < keys) warp.template round<kQueries>(x, at);
            else if (at < values) warp.template round<kKeys>(x, at - keys);
            else warp.template round<kValues>(x, at - values);
        }
        fresh = ++at == upto;
        if (fresh) {
            at = from;
            token += step;
        }
    }
    copies_wait<0>();
}

template <int IO, bool F8, int LANES, int NP> static cudaError_t launch(const RotateArgs &a, int32_t sms, cudaStream_t stream) {
    // A token's heads go to `parts` warps, so that a few tokens have the whole GPU and many end together; but what a warp does for a token
    // (its slot, sines and weights) takes as long as three rounds, and each of them does it again. The time is that of the warp with
    // the most parts. 8192 tokens of 20 rounds in 1 part 58.6 us, in 2 55.0; 2000 in 1 16.3, in 4 21, in 7 25; 600 in 4 6.9, in 8 8.6; 8192 of 4 rounds in
    // 1 19.0, in 2 20.6; 1158 latents of 17 rounds in 1 14.5, in 2 17.2, in 7 27.9.
    const int at_once = 32 / LANES, q_rounds = (a.n_q_heads + at_once - 1) / at_once, kv_rounds = (a.n_kv_heads + at_once - 1) / at_once;
    const int64_t room = (NP == 1 ? 2 : 1) * sms, tokens = (a.n_tokens + kRotateWarps - 1) / kRotateWarps;
    const int64_t rounds = q_rounds + a.planes * kv_rounds;
    int64_t parts = 1;
    double least = 0;
    for (int64_t p = 1; p <= std::min<int64_t>(rounds, room); ++p) {
        const int64_t across = std::min(tokens, room / p) * kRotateWarps;      // tokens at a time
        const double time = (double)((a.n_tokens + across - 1) / across) * (3 + (double)((rounds + p - 1) / p));
        if (p == 1 || time < least) least = time, parts = p;
    }
    dim3 grid((unsigned)std::min(tokens, room / parts), (unsigned)parts);
    // Of wide heads, more tokens than warps: one line of all rounds, of which every warp has as much (5000 latents of 25 rounds 70 us, 86 by whole
    // tokens; 1158 of 17 15.0, 14.4; 300 7.9, 6.8). Not of others: warps then work on rows far apart, which the memory answers more slowly (8192 tokens of 20
    // rounds 61 us for 55).
    RotateArgs args = a;
    args.line = NP > 1 && (double)a.n_tokens * (rounds + 3) / (room * kRotateWarps) + 3 < 0.92 * least;
    if (args.line) grid = dim3((unsigned)room);
    const bool full = a.head_dim == 16 * LANES && a.turned == a.head_dim && (a.norm_dim == a.head_dim || (!a.q_weight && !a.k_weight));
    constexpr int bytes = kRotateWarps * Rotate<IO, F8, LANES, NP, false, false>::RING;
    auto start = [&](auto *kernel, std::atomic<uint64_t> &asked) {
        const cudaError_t e = allow_shared(kernel, bytes, a.device, asked);
        return e != cudaSuccess ? e : launch_after(kernel, grid, kRotateThreads, bytes, stream, args);
    };
    static std::atomic<uint64_t> asked[4];
    if constexpr (NP == 1)
        if (full)
            return a.pairs ? start(kvx_rotate_kernel<IO, F8, LANES, NP, true, true>, asked[0]) : start(kvx_rotate_kernel<IO, F8, LANES, NP, false, true>, asked[1]);
    return a.pairs ? start(kvx_rotate_kernel<IO, F8, LANES, NP, true, false>, asked[2]) : start(kvx_rotate_kernel<IO, F8, LANES, NP, false, false>, asked[3]);
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
