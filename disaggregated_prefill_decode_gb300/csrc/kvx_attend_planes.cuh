// kvx_cache_attend over separate key and value planes: the kernel, instantiated per value type in
// kvx_attend_*.cu (latents: kvx_latent.cu, kvx_latent_tensor.cu).
//
// The softmax runs once over the positions with a running maximum m and sum l per query:
//   m' = max(m, s), l' = l 2^(m - m') + 2^(s - m'), O' = O 2^(m - m') + 2^(s - m') v,
// scores in units of log2, all of it in 32 bits (with f16 products m' = max(m, s - 15): Shape::UP). Bound by memory: each key and value is used by the queries
// of one KV head only, 2 group flops per element, so all that counts is bytes in flight and what a call
// costs before its first and after its last byte.
//
// A warp works alone on its stretch of tiles, with a ring of tiles (keys and values of 16 or 32 positions)
// in shared memory that asynchronous copies fill. S^T = K Q^T takes 16 bytes of a key row as the k
// elements that a lane gives to the products (the queries are loaded in the same order of elements), and
// O^T = V^T P^T takes the bytes of two neighbouring positions interleaved, so every lane reads the ring in
// pieces of 16 bytes and the pieces are swizzled for that alone. Both products have the 8 queries as their
// narrow side, so a group of up to 8 query heads wastes nothing that the memory would wait for, and the
// warp products (mma.sync) are at 16 % of their rate: the tensor pipe of a whole CTA would have 8 of 128
// rows to do.
//
// What it measured on GB300 (8 KV heads of 128, 8 queries each, bf16): 256 requests of 4608 positions 728
// us, 6.6 TB/s, 0.98 of the copy rate; 16 requests of 1024 to 8192 57.4 us, of which 45 are the stream at
// 0.99 of it. Steps on the way: keys and values straight from global memory into registers 125 us (128
// registers a thread were too few: spills); through rings that each lane filled for itself, 64 bytes of a
// row an instruction, 75 (256 requests: 953); whole 128-byte lines and this swizzle 61 (745): the requests
// of half lines had been the limit. 8, 12 and 16 warps a CTA are alike in time; 8 have room for the rings.
#pragma once

#include "kvx_attend.cuh"
#include "kvx_shared_plan.cuh"

namespace kvx {

constexpr int kSharedBytes = 226 << 10;       // of a CTA, one per SM
// What the change to another segment costs a warp, in tiles: outputs, then queries. 200 requests with a window of 1024: 47.8 us
// with 0, 42.1 with 1, 41.6 with 2; long segments the same with all three.
constexpr int kSwitchTiles = 2;
constexpr int kJoinAtOnce = 24;               // pieces of a segment that a warp's join loads at once

template <int VT_, int IO_, int D_, int NT_, bool FULL_> struct Shape {
    static constexpr int VT = VT_, IO = IO_, D = D_, NT = NT_;   // D: head_dim rounded up; NT: query sets of 8
    static constexpr bool FULL = FULL_;                           // head_dim is D
    static constexpr bool REST = false;                           // see RestShape
    using Args = AttendArgs;
    __host__ __device__ static const AttendArgs &attend(const Args &x) { return x; }
    static constexpr bool F8 = VT == KVX_E4M3;
    static constexpr int MT = F8 ? KVX_F16 : VT;                  // type of the products
    // f16 weights are taken times 2^15, by a reference m that far below the maximum: one of 2^-39 of the largest still has a
    // step of f16. Times 1, those below 2^-25 were lost from the outputs (not from the sum), and 2^-14 had no second value.
    static constexpr float UP = MT == KVX_F16 ? 15.0f : 0.0f;
    // A weight is the sum of PARTS values of the products' type. An infinite element of V has to meet neither a zero nor a
    // negative one, which would make it NaN: so with 16-bit planes all but the last are cut off, not rounded, and each is at
    // least LEAST (or the weight). What is left of a weight: f16 2^-22, or 2^-39 of the largest; bf16 2^-22 (two values: 2^-16,
    // which showed in the outputs' rounding); 8-bit codes are finite, their weights' values rounded: 2^-23.
    static constexpr float LEAST = MT == KVX_F16 ? 0x1p-24f : 0x1p-126f;
    static constexpr int PARTS = MT == KVX_F16 ? 2 : 3;
    static constexpr int ESZ = F8 ? 1 : 2;
    static constexpr int TOK = D * ESZ <= 128 ? 32 : 16;          // positions of a tile
    static constexpr int SUB = TOK / 16;
    static constexpr int KCH = D * ESZ / 64;                      // 64-byte chunks of a key row, 16 bytes a lane
    static constexpr int KSTEP = F8 ? 4 : 2;                      // products per chunk
    static constexpr int PIECE = D * ESZ / 8 < 16 ? 8 : 16;       // bytes of a value row a lane copies at once
    static constexpr int NP = D * ESZ / 8 / PIECE;
    static constexpr int PE = PIECE / ESZ;
    static constexpr int NE = D / 8;                              // value elements of a lane
    static constexpr int F4 = D / 16;                             // partial sums of a query set: float4 per lane
    static constexpr int PARTIAL = NT * (F4 * 32 * 16 + 2 * 8 * 4);   // bytes of a partial result: O, m, l
    static constexpr int WARPS = D > 128 ? 4 : 8;                 // of the CTA, 255 registers a thread
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int RP = D * ESZ / 16;                       // 16-byte pieces of a row
    static constexpr int PLANE = TOK * D * ESZ, STAGE = 2 * PLANE;   // a tile: keys, then values
    static constexpr int ROOM = kSharedBytes / WARPS;
    static constexpr bool SLOT = (ROOM - PARTIAL) / STAGE >= 3;   // room for a partial result beside the ring
    static constexpr int STAGES = (ROOM - (SLOT ? PARTIAL : 0)) / STAGE < 6 ? (ROOM - (SLOT ? PARTIAL : 0)) / STAGE : 6;
    static constexpr int RING = STAGES * STAGE, WARP_BYTES = RING + (SLOT ? PARTIAL : 0);
    static_assert(STAGES >= 3 && RING >= PARTIAL, "a warp's last partial result reuses its ring");
    // places of a 16-byte piece of a row, and of the 16 (8) bytes that lane (g, t) takes, in a plane of a tile
    static __device__ __forceinline__ uint32_t key_at(int u, int c, int h, int g, int t) {
        return ((u * KCH + c) * 2 + h) * 512 + (((g * 4 + t) ^ (c & 1) * 4)) * 16;
    }
    static __device__ __forceinline__ uint32_t value_at(int u, int j, int c, int g, int t) {
        if constexpr (PIECE == 16) return ((u * 4 + j) * NP + c) * 512 + (t * 8 + (g ^ t * 2)) * 16;
        else return (u * 4 + j) * 256 + t * 64 + (g / 2 ^ t / 2 * 2) * 16 + g % 2 * 8;
    }
    // value elements 2e and 2e + 1 of a lane in row group g are rows g and g + 8 of product e
    static __device__ __forceinline__ int dim(int g, int e) { return e / PE * (8 * PE) + g * PE + e % PE; }
};

// The positions of requests behind the prefixes that kvx_cache_attend_shared has taken: in the place of outputs, sums in 32 bits
// that its last kernel joins with those of the prefixes. It also joins what several CTAs have of a segment, so none waits for another's.
template <class S> struct RestShape : S {
    static constexpr bool REST = true;
    static_assert(S::WARPS * S::WARP_BYTES + kRestFew * 4 + 512 <= (227 << 10), "beside the rings there is room for kRestFew requests");
    using Args = SharedArgs;
    __host__ __device__ static const AttendArgs &attend(const Args &x) { return x.a; }
};

// A partial result in shared memory or in the scratch: O as [set][query of the lane's two][e / 4][lane] float4 of four
// value elements, then m and l of the queries.
template <class S> struct Partial {
    float4 *o;
    float *m, *l;
    __device__ __forceinline__ explicit Partial(uint8_t *p)
        : o((float4 *)p), m((float *)(p + S::NT * S::F4 * 512)), l(m + 8 * S::NT) {}
};

template <class S>
__device__ __forceinline__ void write_lse(const AttendArgs &a, int32_t r, int32_t head, float m, float l) {
    if (a.lse) a.lse[(int64_t)r * a.n_q_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Partial results to join: one, and those at equal distances.
struct Pieces {
    uint8_t *first, *others;
    int step, n;
    __device__ __forceinline__ uint8_t *at(int x) const { return x ? others + x * step : first; }
};

// What one lane has of a join: float4 f of the sums, for query q.
template <class S> struct Joined {
    int f, q, e4;
    float top, l;
    float4 o;
    __device__ __forceinline__ explicit Joined(int f_) : f(f_), top(-INFINITY), l(0.0f), o(make_float4(0, 0, 0, 0)) {
        const int t = threadIdx.x & 3, i = f % S::F4 / (S::F4 / 2);
        e4 = f % (S::F4 / 2);
        q = f / S::F4 * 8 + 2 * t + i;
    }
    // Into another partial result, or, without one, the outputs.
    __device__ __forceinline__ void put(const AttendArgs &a, uint8_t *to, int32_t r, int32_t head0, int32_t heads) const {
        const int lane = threadIdx.x & 31, g = lane >> 2;
        if (!to) {
            const int d = S::dim(g, e4 * 4);
            if (q < heads && (S::FULL || d < a.head_dim)) {
                const float inv = l == 0.0f ? 0.0f : a.v_scale / l;
                const uint2 y = make_uint2(pack<S::IO>(o.x * inv, o.y * inv), pack<S::IO>(o.z * inv, o.w * inv));
                *reinterpret_cast<uint2 *>(a.out + r * a.out_stride + ((int64_t)(head0 + q) * a.head_dim + d) * 2) = y;
            }
            if (q < heads && e4 == 0 && g == 0) write_lse<S>(a, r, head0 + q, top, l);
        } else {
            const Partial<S> p(to);
            __stcg(p.o + f * 32 + lane, o);
            if (e4 == 0 && g == 0) {
                __stcg(p.m + q, top);
                __stcg(p.l + q, l);
            }
        }
    }
    // REST: the segment's sums, of which `more` CTAs behind this one have more, or (begun) what this CTA adds to another one's.
    __device__ __forceinline__ void put_rest(const AttendArgs &a, bool begun, int32_t more, int32_t r, int32_t head0, int32_t heads) const {
        const int g = (threadIdx.x & 31) >> 2, d = S::dim(g, e4 * 4);
        if (q >= heads) return;
        const int64_t row = (int64_t)r * a.n_q_heads + head0 + q;
        uint8_t *const part = a.rest_parts + blockIdx.x * rest_part_bytes(a.head_dim);
        float *const to = begun ? reinterpret_cast<float *>(part + kRestRows * 8) + q * a.head_dim : a.rest + row * a.head_dim;
        if (S::FULL || d < a.head_dim) *reinterpret_cast<float4 *>(to + d) = o;
        if (e4 != 0 || g != 0) return;
        if (begun) reinterpret_cast<float2 *>(part)[q] = make_float2(top, l);
        else a.rest_ml[row] = make_float4(top, l, __int_as_float((int32_t)blockIdx.x + 1), __int_as_float(more));
    }
};

// One warp: float4 f of a few partial results of this CTA's warps, or (SCRATCH) of other CTAs, which come from L2.
template <class S, bool SCRATCH>
__device__ __forceinline__ Joined<S> join_few(int f, const Pieces &from) {
    constexpr int AT_ONCE = 4;
    Joined<S> j(f);
    auto get = [](const auto *p) {
        if constexpr (SCRATCH) return __ldcg(p);
        else return *p;
    };
    for (int x0 = 0; x0 < from.n; x0 += AT_ONCE) {
        float4 y[AT_ONCE];
        float m[AT_ONCE], l[AT_ONCE], up = j.top;
#pragma unroll
        for (int x = 0; x < AT_ONCE; ++x) {
            m[x] = -INFINITY;
            if (x0 + x < from.n) {
                const Partial<S> p(from.at(x0 + x));
                y[x] = get(p.o + f * 32 + (threadIdx.x & 31));
                m[x] = get(p.m + j.q);
                l[x] = get(p.l + j.q);
            }
        }
#pragma unroll
        for (int x = 0; x < AT_ONCE; ++x) up = fmaxf(up, m[x]);
        const float ref = up == -INFINITY ? 0.0f : up, old = fast_exp2(j.top - ref);
        j.top = up;
        j.l *= old;
        j.o = make_float4(j.o.x * old, j.o.y * old, j.o.z * old, j.o.w * old);
#pragma unroll
        for (int x = 0; x < AT_ONCE; ++x)
            if (x0 + x < from.n) {
                const float w = fast_exp2(m[x] - ref);
                j.l += w * l[x];
                j.o.x += w * y[x].x;
                j.o.y += w * y[x].y;
                j.o.z += w * y[x].z;
                j.o.w += w * y[x].w;
            }
    }
    return j;
}

// The same of many in the scratch, kJoinAtOnce at once: lane (g, t) takes the maxima and sums of every eighth for its query, the others'
// weights come by shuffles.
template <class S> __device__ __noinline__ Joined<S> join_many(int f, const Pieces &from) {
    constexpr int ROUNDS = kJoinAtOnce / 8;
    const int lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2, n = from.n;
    Joined<S> j(f);
    for (int x0 = 0; x0 < n; x0 += 8 * ROUNDS) {
        float4 y[ROUNDS][8];
        float m[ROUNDS], s[ROUNDS], up = j.top;
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            const int x = x0 + 8 * k + g;
            const Partial<S> p(from.at(min(x, n - 1)));
            m[k] = x < n ? __ldcg(p.m + j.q) : -INFINITY;
            s[k] = x < n ? __ldcg(p.l + j.q) : 0.0f;
            if (x0 + 8 * k < n) {
#pragma unroll
                for (int x = 0; x < 8; ++x) y[k][x] = __ldcg(Partial<S>(from.at(min(x0 + 8 * k + x, n - 1))).o + f * 32 + lane);
            }
        }
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) up = fmaxf(up, m[k]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) up = fmaxf(up, __shfl_xor_sync(~0u, up, d));
        const float ref = up == -INFINITY ? 0.0f : up, old = fast_exp2(j.top - ref);
        j.top = up;
        j.l *= old;
        j.o = make_float4(j.o.x * old, j.o.y * old, j.o.z * old, j.o.w * old);
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k)
            if (x0 + 8 * k < n) {
                const float mine = fast_exp2(m[k] - ref);
                j.l += mine * s[k];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float w = __shfl_sync(~0u, mine, x * 4 + t);
                    if (x0 + 8 * k + x < n) {                      // not the last one again: 0 times infinity
                        j.o.x += w * y[k][x].x;
                        j.o.y += w * y[k][x].y;
                        j.o.z += w * y[k][x].z;
                        j.o.w += w * y[k][x].w;
                    }
                }
            }
    }
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) j.l += __shfl_xor_sync(~0u, j.l, d);
    return j;
}

// Offset, in 16-byte units, of the position `lane` of a tile in its buffer; kNoRow for a position that is left out. In two
// steps, so that other loads can start before the block id is waited for.
template <int TOK, class Line> struct Row {
    uint32_t rest;                                                 // within the block, in 16-byte units
    int32_t blk;                                                   // -2: no live position
    __device__ __forceinline__ Row(const AttendArgs &a, const Line &p) : rest(0), blk(-2) {
        const int lane = threadIdx.x & 31;
        const uint32_t pos = (uint32_t)p.first / TOK * TOK + (uint32_t)p.tile * TOK + lane;
        if (lane >= TOK || pos < (uint32_t)p.first || pos >= (uint32_t)p.len) return;
        const uint32_t col = (__umulhi(pos, a.block_mul) + pos) >> a.block_shift;
        blk = max(a.block_table[p.r * a.table_stride + col], -1);
        rest = (pos - col * (uint32_t)a.pool.block_size) * a.token_pitch16;
    }
    __device__ __forceinline__ uint32_t offset(const AttendArgs &a, bool report) const {
        if (blk >= 0 && blk < a.pool.n_blocks) return (uint32_t)blk * a.block_pitch16 + rest;
        if (blk != -2 && report) atomicAdd(a.pool.skipped, 1ull);
        return kNoRow;
    }
};

template <class S> __global__ void __launch_bounds__(S::THREADS, 1) kvx_attend_planes(const __grid_constant__ typename S::Args args) {
    const AttendArgs &a = S::attend(args);
    constexpr int TOK = S::TOK, NT = S::NT;
    using Line = Place<TOK, kSwitchTiles, S::REST>;
    extern __shared__ __align__(16) uint8_t smem[];                // [warp] ring and partial result
    __shared__ int64_t s_seg[S::WARPS][2];                     // first tile of each one's segment; -1: none
    __shared__ int32_t s_where[S::WARPS][2][3];                // request, segment of the request, tiles
    __shared__ int32_t s_pieces[2], s_from[2];                 // of the open segments that this CTA has to join, and the first CTA
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int32_t group = a.n_q_heads / a.n_kv_heads, sets = (group + 8 * NT - 1) / (8 * NT), segs = a.n_kv_heads * sets;

    wait_for_earlier();
    if constexpr (S::REST)
        if (!a.start && plan_few<S::THREADS>(args, smem)) return;
    const Batch<TOK, S::WARPS, S::WARPS, kSwitchTiles, kJoinAtOnce, S::REST> batch(a, segs);
    const Split &split = batch.split;
    if ((int32_t)blockIdx.x >= split.ctas) return;
    uint32_t *const arrived = (uint32_t *)a.scratch;
    uint8_t *const cta_parts = a.scratch + kScratchCounters * sizeof(uint32_t);             // [CTA][2]
    const int64_t c_begin = split.begin(blockIdx.x), c_end = split.begin(blockIdx.x + 1);
    auto first_slot = [&](int warp) {
        return S::SLOT ? smem + warp * S::WARP_BYTES + S::RING : cta_parts + (size_t)(2 * gridDim.x + blockIdx.x * S::WARPS + warp) * S::PARTIAL;
    };
    const int64_t per = (c_end - c_begin) / S::WARPS, more = (c_end - c_begin) % S::WARPS;   // warps without work come last
    int64_t x0 = c_begin + w * per + min((int64_t)w, more);
    const int64_t x1 = x0 + per + (w < more);
    if (lane < 2) s_seg[w][lane] = -1;
    __syncwarp();

    if (x0 < x1) {
        const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem + w * S::WARP_BYTES);
        uint32_t q[NT][S::KCH * S::KSTEP][2];
        float o[NT][S::NE / 2][4], m[NT][2], l[NT][2], sc[NT][2];
        Line cur = batch.locate(a, segs, x0), far = cur;
        const uint8_t *k_ptr, *v_ptr;                              // this lane's piece of row 0 of the head
        constexpr int RI = 32 / S::RP;                             // rows that a copy of the warp covers
        const int piece = lane % S::RP;
        const bool piece_in = S::FULL || piece * 16 < a.head_dim * S::ESZ;

        auto pointers = [&](const Line &p) {
            const int32_t kvh = p.seg / sets, shard = kvh / a.pool.heads_per_shard;
            const int64_t off = (int64_t)(kvh - shard * a.pool.heads_per_shard) * a.pool.head_pitch;
            k_ptr = a.pool.k[shard] + off + piece * 16;
            v_ptr = a.pool.v[shard] + off + piece * 16;
        };
        auto load_tile = [&](uint32_t row, uint32_t to) {
#pragma unroll
            for (int i = 0; i < TOK / RI; ++i) {
                const int x = i * RI + lane / S::RP, y = x % 16;   // row of the tile
                const uint32_t at = __shfl_sync(~0u, row, x);
                const uint64_t off = at == kNoRow ? 0 : (uint64_t)at * 16;
                const bool in = at != kNoRow && piece_in;
                copy_async(to + S::key_at(x / 16, piece / 4, y / 8, y % 8, piece % 4), k_ptr + off, in);
                const int g = S::PIECE == 16 ? piece % 8 : piece * 2;
                copy_async(to + S::PLANE + S::value_at(x / 16, (y & 1) + y / 8 * 2, piece / 8, g, y % 8 / 2), v_ptr + off, in);
            }
            copies_commit();
        };
        // Queries of a segment. 8-bit caches multiply in f16: a bf16 row is brought by a power of two to where f16 holds
        // its elements exactly down to 2^-31 of the largest.
        auto load_q = [&](const Line &p) {
            const int32_t kvh = p.seg / sets, first = p.seg % sets * 8 * NT;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int32_t qi = first + n * 8 + g;
                const uint8_t *src = a.q + p.r * a.q_stride + ((int64_t)kvh * group + qi) * a.head_dim * 2;
#pragma unroll
                for (int c = 0; c < S::KCH; ++c)
#pragma unroll
                    for (int h = 0; h < S::KSTEP / 2; ++h) {
                        const int d = (c * 64 + t * 16) / S::ESZ + h * 8;
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if (qi < group && (S::FULL || d < a.head_dim)) x = __ldg(reinterpret_cast<const uint4 *>(src + d * 2));
                        uint32_t *y = &q[n][c * S::KSTEP + h * 2][0];
                        y[0] = x.x;
                        y[1] = x.y;
                        y[2] = x.z;
                        y[3] = x.w;
                    }
                float scale = a.scale;
                if constexpr (S::F8 && S::IO == KVX_BF16) {
                    uint32_t *y = &q[n][0][0];
                    float top = 0.0f;
#pragma unroll
                    for (int i = 0; i < S::KCH * S::KSTEP * 2; ++i) {
                        const float2 f = unpack<KVX_BF16>(y[i]);
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                    const int e = top > 0.0f && top < INFINITY ? max(-126, min(100, 14 - ilogbf(top))) : 0;
                    const float up = __int_as_float((127 + e) << 23);
                    scale = fmaxf(scale * __int_as_float((127 - e) << 23), kLeastScale);
#pragma unroll
                    for (int i = 0; i < S::KCH * S::KSTEP * 2; ++i) {
                        const float2 f = unpack<KVX_BF16>(y[i]);
                        y[i] = pack<KVX_F16>(f.x * up, f.y * up);
                    }
                }
                sc[n][0] = __shfl_sync(~0u, scale, 8 * t);         // of queries 2t and 2t + 1
                sc[n][1] = __shfl_sync(~0u, scale, 8 * t + 4);
                m[n][0] = m[n][1] = -INFINITY;
                l[n][0] = l[n][1] = 0.0f;
#pragma unroll
                for (int e = 0; e < S::NE / 2; ++e) o[n][e][0] = o[n][e][1] = o[n][e][2] = o[n][e][3] = 0.0f;
            }
        };
        // The end of this warp's part of a segment, [from, to) of the line: outputs if it is the whole of it, else a partial result.
        auto flush = [&](const Line &p, int64_t from, int64_t to) {
            const int64_t begin = p.seg_begin(segs);
            const int32_t kvh = p.seg / sets, first = p.seg % sets * 8 * NT;
            const bool whole = from == begin && to == begin + p.tiles;
            const int slot = from == begin;                        // 1: the warp's last, with nothing left in its ring
            if (!whole && lane == 0) {
                s_seg[w][slot] = begin;
                s_where[w][slot][0] = p.r;
                s_where[w][slot][1] = p.seg;
                s_where[w][slot][2] = p.tiles;
            }
            const Partial<S> part(slot ? smem + w * S::WARP_BYTES : first_slot(w));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[n][i] += __shfl_xor_sync(~0u, l[n][i], d);
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int32_t qi = first + n * 8 + 2 * t + i, head = kvh * group + qi;
                        if (qi >= group) continue;
                        if constexpr (S::REST) {
                            const int64_t row = (int64_t)p.r * a.n_q_heads + head;
#pragma unroll
                            for (int e = 0; e < S::NE / 2; e += 2) {
                                const int d = S::dim(g, 2 * e);
                                if (S::FULL || d < a.head_dim)
                                    *reinterpret_cast<float4 *>(a.rest + row * a.head_dim + d) =
                                        make_float4(o[n][e][i], o[n][e][2 + i], o[n][e + 1][i], o[n][e + 1][2 + i]);
                            }
                            if (g == 0) a.rest_ml[row] = make_float4(m[n][i], l[n][i], 0.0f, 0.0f);
                            continue;
                        }
                        const float inv = l[n][i] == 0.0f ? 0.0f : a.v_scale / l[n][i];
                        uint8_t *dst = a.out + p.r * a.out_stride + (int64_t)head * a.head_dim * 2;
#pragma unroll
                        for (int e = 0; e < S::NE / 2; e += 2) {
                            const int d = S::dim(g, 2 * e);
                            if (S::FULL || d < a.head_dim)
                                *reinterpret_cast<uint2 *>(dst + d * 2) = make_uint2(pack<S::IO>(o[n][e][i] * inv, o[n][e][2 + i] * inv),
                                                                                     pack<S::IO>(o[n][e + 1][i] * inv, o[n][e + 1][2 + i] * inv));
                        }
                        if (g == 0) write_lse<S>(a, p.r, head, m[n][i], l[n][i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < S::NE / 2; e += 2)
                            part.o[((n * 2 + i) * (S::F4 / 2) + e / 2) * 32 + lane] =
                                make_float4(o[n][e][i], o[n][e][2 + i], o[n][e + 1][i], o[n][e + 1][2 + i]);
                    if (g == 0)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            part.m[n * 8 + 2 * t + i] = m[n][i];
                            part.l[n * 8 + 2 * t + i] = l[n][i];
                        }
                }
            }
        };

        // rows[n]: offsets of the tile n after this one; `far` is the tile AHEAD after this one, the next to be copied.
        constexpr int AHEAD = S::STAGES - 1;
        uint32_t rows[AHEAD + 1];
        int64_t far_x = x0;
        pointers(far);
#pragma unroll
        for (int n = 0; n < AHEAD; ++n) {
            rows[n] = kNoRow;
            if (far_x < x1) {
                const Row<TOK, Line> row(a, far);
                if (n == 0 && !S::F8) load_q(cur);                 // 8-bit caches' queries are waited for, so after the copies
                else if (n && far.tile == 0) pointers(far);
                rows[n] = row.offset(a, far.seg == 0);
                load_tile(rows[n], ring + n * S::STAGE);
                far.next(a, segs, far_x);
            } else copies_commit();
        }
        if (S::F8 && x0 < x1) load_q(cur);
        int64_t from = x0;
        int stage = 0, free_stage = AHEAD;
        for (int64_t x = x0; x < x1;) {
            const bool ahead = far_x < x1;
            rows[AHEAD] = ahead ? Row<TOK, Line>(a, far).offset(a, far.seg == 0) : kNoRow;
            copies_wait<AHEAD - 1>();
            __syncwarp();                                          // lanes read what others copied; all are done with free_stage
            if (ahead) {
                if (far.tile == 0) pointers(far);
                load_tile(rows[AHEAD], ring + free_stage * S::STAGE);
                far.next(a, segs, far_x);
            } else copies_commit();
            const uint32_t keys = ring + stage * S::STAGE, values = keys + S::PLANE;
            float s[NT][S::SUB][4];
#pragma unroll
            for (int u = 0; u < S::SUB; ++u) {
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n][u][0] = s[n][u][1] = s[n][u][2] = s[n][u][3] = 0.0f;
#pragma unroll
                for (int c = 0; c < S::KCH; ++c) {
                    uint32_t k[2][4];
                    shared_read(k[0], keys + S::key_at(u, c, 0, g, t));
                    shared_read(k[1], keys + S::key_at(u, c, 1, g, t));
#pragma unroll
                    for (int i = 0; i < S::KSTEP; ++i) {
                        uint32_t a0, a1, a2, a3;
                        if constexpr (S::F8) {
                            f16_of_codes(k[0][i], a0, a2);
                            f16_of_codes(k[1][i], a1, a3);
                        } else {
                            a0 = k[0][2 * i], a2 = k[0][2 * i + 1], a1 = k[1][2 * i], a3 = k[1][2 * i + 1];
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma<S::MT>(s[n][u], a0, a1, a2, a3, q[n][c * S::KSTEP + i][0], q[n][c * S::KSTEP + i][1]);
                    }
                }
            }
            uint32_t parts[S::PARTS][NT][S::SUB][2];
            if (__any_sync(~0u, lane < TOK && rows[0] == kNoRow)) {
#pragma unroll
                for (int u = 0; u < S::SUB; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (__shfl_sync(~0u, rows[0], u * 16 + h * 8 + g) == kNoRow)
#pragma unroll
                            for (int n = 0; n < NT; ++n) s[n][u][2 * h] = s[n][u][2 * h + 1] = -INFINITY;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float old[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float top = fmaxf(s[n][0][i], s[n][0][2 + i]);
#pragma unroll
                    for (int u = 1; u < S::SUB; ++u) top = fmaxf(top, fmaxf(s[n][u][i], s[n][u][2 + i]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                    top = fmaxf(m[n][i], fmaf(top, sc[n][i], -S::UP));
                    const float ref = top == -INFINITY ? 0.0f : top;
                    old[i] = fast_exp2(m[n][i] - ref);
                    m[n][i] = top;
                    l[n][i] *= old[i];
#pragma unroll
                    for (int u = 0; u < S::SUB; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float p = fast_exp2(fmaf(s[n][u][2 * h + i], sc[n][i], -ref));
                            s[n][u][2 * h + i] = p;
                            l[n][i] += p;
                        }
                }
                if (__any_sync(~0u, old[0] != 1.0f || old[1] != 1.0f)) {
#pragma unroll
                    for (int e = 0; e < S::NE / 2; ++e) {
                        o[n][e][0] *= old[0];
                        o[n][e][1] *= old[1];
                        o[n][e][2] *= old[0];
                        o[n][e][3] *= old[1];
                    }
                }
#pragma unroll
                for (int u = 0; u < S::SUB; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float p0 = s[n][u][2 * h], p1 = s[n][u][2 * h + 1];
                        const float least0 = fminf(p0, S::LEAST), least1 = fminf(p1, S::LEAST);
#pragma unroll
                        for (int k = 0; k < S::PARTS; ++k) {
                            const uint32_t x = S::F8 || k + 1 == S::PARTS ? pack<S::MT>(p0, p1) : pack_down<S::MT>(p0, p1);
                            parts[k][n][u][h] = transpose8x8(x);
                            const float2 f = unpack<S::MT>(x);
                            p0 = S::F8 ? p0 - f.x : fmaxf(p0 - f.x, least0);
                            p1 = S::F8 ? p1 - f.y : fmaxf(p1 - f.y, least1);
                        }
                    }
            }
#pragma unroll
            for (int u = 0; u < S::SUB; ++u)
#pragma unroll
                for (int c = 0; c < S::NP; ++c) {
                    uint32_t v[4][S::PIECE / 4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        shared_read(v[j], values + S::value_at(u, j, c, g, t));
                    uint32_t av[S::PE / 2][4];                      // element 2e, element 2e + 1; the same 8 positions on
#pragma unroll
                    for (int e = 0; e < S::PE / 2; ++e)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if constexpr (S::F8) {
                                const uint32_t x = __byte_perm(v[2 * j][e / 2], v[2 * j + 1][e / 2], e & 1 ? 0x7362 : 0x5140);
                                f16_of_codes(x, av[e][2 * j], av[e][2 * j + 1]);
                            } else {
                                av[e][2 * j] = __byte_perm(v[2 * j][e], v[2 * j + 1][e], 0x5410);
                                av[e][2 * j + 1] = __byte_perm(v[2 * j][e], v[2 * j + 1][e], 0x7632);
                            }
                        }
#pragma unroll
                    for (int k = 0; k < S::PARTS; ++k)
#pragma unroll
                        for (int e = 0; e < S::PE / 2; ++e)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma<S::MT>(o[n][c * (S::PE / 2) + e], av[e][0], av[e][1], av[e][2], av[e][3], parts[k][n][u][0], parts[k][n][u][1]);
                }
            const bool ends = cur.tile + 1 == cur.tiles;
            const int64_t here = x;
            Line nxt = cur;
            nxt.next(a, segs, x);
            if (ends || x >= x1) {
                flush(cur, from, here + 1);
                from = x;
                if (x >= x1) break;
                load_q(nxt);
            }
            cur = nxt;
#pragma unroll
            for (int n = 0; n < AHEAD; ++n) rows[n] = rows[n + 1];
            free_stage = stage;
            stage = stage + 1 == S::STAGES ? 0 : stage + 1;
        }
    }
    __syncthreads();

    // Segments whose pieces several warps hold, in order: the second of one warp, the first ones of those after it. Each warp joins
    // some float4s of some of them. At most two go on in other CTAs: one that began before this one's stretch, one that ends after it.
    auto heads_of = [&](int32_t seg, int32_t *head0) {
        const int32_t first = seg % sets * 8 * NT;
        *head0 = seg / sets * group + first;
        return min(group - first, 8 * NT);
    };
    constexpr int FS = NT * S::F4;
    static_assert(2 * S::WARPS <= 32, "a lane per piece");
    const int64_t my_seg = lane < 2 * S::WARPS ? s_seg[lane >> 1][lane & 1] : -1;
    const uint32_t pieces = __ballot_sync(~0u, my_seg >= 0), lower = pieces & ((1u << lane) - 1);
    const int64_t prev_seg = __shfl_sync(~0u, my_seg, lower ? 31 - __clz(lower) : lane);
    const bool leads = my_seg >= 0 && (!lower || prev_seg != my_seg);
    uint32_t leaders = __ballot_sync(~0u, leads);                  // the first piece of each segment
    int my_open = 0;                                               // 1: begun before, 2: goes on after this CTA
    if (leads) my_open = my_seg < c_begin ? 1 : my_seg + s_where[lane >> 1][lane & 1][2] > c_end ? 2 : 0;
    const uint32_t open1 = __ballot_sync(~0u, my_open == 1), open2 = __ballot_sync(~0u, my_open == 2);
    const int open[2] = {__ffs(open1) - 1, __ffs(open2) - 1};
    for (int task = w; leaders; task -= FS, leaders &= leaders - 1) {
        if (task >= FS) continue;
        const int i = __ffs(leaders) - 1;
        const uint32_t rest = leaders & (leaders - 1);
        const int n = __popc(pieces & (rest ? (1u << (__ffs(rest) - 1)) - 1 : ~0u) & ~((1u << i) - 1));
        const int32_t *where = s_where[i >> 1][i & 1];
        int32_t head0;
        const int32_t heads = heads_of(where[1], &head0);
        uint8_t *const first = i & 1 ? smem + (i >> 1) * S::WARP_BYTES : first_slot(i >> 1);
        const Pieces from = {first, first_slot(i >> 1), S::SLOT ? S::WARP_BYTES : S::PARTIAL, n};
        if constexpr (S::REST) {                                   // the pieces of other CTAs are joined with the prefix
            const int32_t more = i == open[1] ? split.cta_of(s_seg[i >> 1][i & 1] + where[2] - 1) - (int32_t)blockIdx.x : 0;
            for (; task < FS; task += S::WARPS) join_few<S, false>(task, from).put_rest(a, i == open[0], more, where[0], head0, heads);
            continue;
        }
        uint8_t *const to = i == open[0] || i == open[1] ? cta_parts + (size_t)(blockIdx.x * 2 + (i == open[1])) * S::PARTIAL : nullptr;
        for (; task < FS; task += S::WARPS) join_few<S, false>(task, from).put(a, to, where[0], head0, heads);
    }
    if (S::REST || (open[0] < 0 && open[1] < 0)) return;
    __syncthreads();
    if (threadIdx.x < 2) {
        const int i = open[threadIdx.x];
        s_pieces[threadIdx.x] = 0;
        if (i >= 0) {
            const int64_t seg = s_seg[i >> 1][i & 1];
            const int32_t from = split.cta_of(seg), upto = split.cta_of(seg + s_where[i >> 1][i & 1][2] - 1);
            // releases what the CTA's threads wrote before the barrier, acquires what the other CTAs' did
            uint32_t before;
            asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(arrived + from) : "memory");
            if (before == (uint32_t)(upto - from)) {
                arrived[from] = 0;                                 // for the next call
                s_pieces[threadIdx.x] = upto - from + 1;
                s_from[threadIdx.x] = from;
            }
        }
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
        const int n = s_pieces[k];
        if (!n) continue;
        const int32_t *where = s_where[open[k] >> 1][open[k] & 1], from = s_from[k];
        int32_t head0;
        const int32_t heads = heads_of(where[1], &head0);
        const Pieces pieces = {cta_parts + (size_t)(2 * from + 1) * S::PARTIAL, cta_parts + (size_t)(2 * from) * S::PARTIAL, 2 * S::PARTIAL, n};
        for (int f = w; f < FS; f += S::WARPS) {
            if (n <= 8) join_few<S, true>(f, pieces).put(a, nullptr, where[0], head0, heads);
            else join_many<S>(f, pieces).put(a, nullptr, where[0], head0, heads);
        }
    }
}

// ------------------------------------------------------------------------------------------------

template <class S> static cudaError_t launch(const typename S::Args &args, int32_t sms, cudaStream_t stream) {
    constexpr int bytes = S::WARPS * S::WARP_BYTES;
    static std::atomic<uint64_t> asked;
    const cudaError_t e = allow_shared(kvx_attend_planes<S>, bytes, S::attend(args).device, asked);
    if (e != cudaSuccess) return e;
    return launch_after(kvx_attend_planes<S>, dim3(sms), S::THREADS, bytes, stream, args);
}

template <int VT, int IO, int D, int NT> static cudaError_t launch(const AttendArgs &a, int32_t sms, cudaStream_t stream) {
    return a.head_dim == D ? launch<Shape<VT, IO, D, NT, true>>(a, sms, stream) : launch<Shape<VT, IO, D, NT, false>>(a, sms, stream);
}

// Head dims are rounded up to 64, 128 or 256; more than 8 query heads to a KV head are taken 16 at a time.
template <int VT, int IO> static cudaError_t launch_planes(const AttendArgs &a, int32_t sms, cudaStream_t stream) {
    const bool wide = a.n_q_heads / a.n_kv_heads > 8;
    if (a.head_dim <= 64) return wide ? launch<VT, IO, 64, 2>(a, sms, stream) : launch<VT, IO, 64, 1>(a, sms, stream);
    if (a.head_dim <= 128) return wide ? launch<VT, IO, 128, 2>(a, sms, stream) : launch<VT, IO, 128, 1>(a, sms, stream);
    return launch<VT, IO, 256, 1>(a, sms, stream);
}

// The same for the rest of requests, head dims up to 128.
template <int VT, int IO, int D, int NT> static cudaError_t launch_rest_shape(const SharedArgs &s, int32_t sms, cudaStream_t stream) {
    return s.a.head_dim == D ? launch<RestShape<Shape<VT, IO, D, NT, true>>>(s, sms, stream) : launch<RestShape<Shape<VT, IO, D, NT, false>>>(s, sms, stream);
}
template <int VT, int IO> static cudaError_t launch_rest_planes(const SharedArgs &s, int32_t sms, cudaStream_t stream) {
    const bool wide = s.a.n_q_heads / s.a.n_kv_heads > 8;
    if (s.a.head_dim <= 64) return wide ? launch_rest_shape<VT, IO, 64, 2>(s, sms, stream) : launch_rest_shape<VT, IO, 64, 1>(s, sms, stream);
    return wide ? launch_rest_shape<VT, IO, 128, 2>(s, sms, stream) : launch_rest_shape<VT, IO, 128, 1>(s, sms, stream);
}

}  // namespace kvx
