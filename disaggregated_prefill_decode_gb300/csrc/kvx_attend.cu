// kvx_cache_attend over separate key and value planes, and its launcher (latents: kvx_latent.cu).
//
// The softmax runs once over the positions with a running maximum m and sum l per query:
//   m' = max(m, s), l' = l 2^(m - m') + 2^(s - m'), O' = O 2^(m - m') + 2^(s - m') v,
// scores in units of log2. Bound by memory: each key and value is used by the queries of one KV head
// only, 2 group flops per element, so all that counts is bytes in flight.
//
// A warp works alone on its stretch of tiles. Keys and values go from global memory straight into the
// registers that feed the matrix products, with no shared memory between: S^T = K Q^T takes a lane's 16
// bytes of a key row as the k elements of the product (the queries are loaded in the same order of
// elements), and O^T = V^T P^T takes the bytes of two neighbouring positions interleaved. Both products
// have the 8 queries as their narrow side, so a group of up to 8 query heads wastes nothing that the
// memory would wait for. K of the next tile is loaded after this tile's scores, V of the next after this
// tile's sums, so that 4 to 8 KB per warp are always on their way.
#include "kvx_attend.cuh"

#include <algorithm>

namespace kvx {

template <int VT_, int IO_, int D_, int NT_> struct Shape {
    static constexpr int VT = VT_, IO = IO_, D = D_, NT = NT_;   // D: head_dim rounded up; NT: query sets of 8
    static constexpr bool F8 = VT == KVX_E4M3;
    static constexpr int MT = F8 ? KVX_F16 : VT;                  // type of the products
    static constexpr int ESZ = F8 ? 1 : 2;
    static constexpr int TOK = D * ESZ <= 128 ? 32 : 16;          // positions of a tile
    static constexpr int SUB = TOK / 16;
    static constexpr int KCH = D * ESZ / 64;                      // 64-byte chunks of a key row, 16 bytes a lane
    static constexpr int KSTEP = F8 ? 4 : 2;                      // products per chunk
    static constexpr int PIECE = D * ESZ / 8 < 16 ? 8 : 16;       // bytes of a value row a lane loads at once
    static constexpr int NP = D * ESZ / 8 / PIECE;
    static constexpr int PE = PIECE / ESZ;
    static constexpr int NE = D / 8;                              // value elements of a lane
    static constexpr int F4 = D / 16;                             // partial sums of a query set: float4 per lane
    static constexpr int PARTIAL = NT * (F4 * 32 * 16 + 2 * 8 * 4);   // bytes of a partial result: O, m, l
    // K, V, O and Q live in registers: 128 suffice for 64 + 32 + 16 of them and leave two CTAs per SM
    static constexpr int CTAS = TOK * D * ESZ <= 4096 && NT * D <= 128 ? 2 : 1;
    // element e of a lane in row group g
    static __device__ __forceinline__ int dim(int g, int e) { return e / PE * (8 * PE) + g * PE + e % PE; }
};

// A partial result in shared memory or in the scratch: O as [set][c][e / 4][lane] float4, where c and e are the place in
// the product's result registers, then m and l of the queries.
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

// Partial results of other CTAs are read from L2, where they were put.
template <bool SCRATCH, class T> __device__ __forceinline__ T read(const T *p) {
    if constexpr (SCRATCH) return __ldcg(p);
    else return *p;
}

// The whole CTA: joins n partial results, `at(i)` the i-th (in the scratch, or in shared memory), into the outputs or into
// another partial result in the scratch.
template <class S, bool SCRATCH, class At>
__device__ __forceinline__ void join(const AttendArgs &a, int n, At at, bool final, uint8_t *to, int32_t r, int32_t head0,
                                     int32_t heads) {
    const int lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
    for (int f = threadIdx.x >> 5; f < S::NT * S::F4; f += kAttendWarps) {
        const int set = f / S::F4, c = f % S::F4 / (S::F4 / 4), e4 = f % (S::F4 / 4);
        const int q = set * 8 + 2 * t + (c & 1);
        float top = -INFINITY;
        for (int i = 0; i < n; ++i) top = fmaxf(top, read<SCRATCH>(Partial<S>(at(i)).m + q));
        const float ref = top == -INFINITY ? 0.0f : top;
        float4 o = make_float4(0, 0, 0, 0);
        float l = 0.0f;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const Partial<S> p(at(i));
            const float w = fast_exp2(read<SCRATCH>(p.m + q) - ref);
            const float4 x = read<SCRATCH>(p.o + f * 32 + lane);
            l += w * read<SCRATCH>(p.l + q);
            o.x += w * x.x;
            o.y += w * x.y;
            o.z += w * x.z;
            o.w += w * x.w;
        }
        if (final) {
            const int d = S::dim(g, (c >> 1) * (S::NE / 2) + e4 * 4);
            if (q < heads && d < a.head_dim) {
                const float inv = l == 0.0f ? 0.0f : a.v_scale / l;
                const uint2 y = make_uint2(pack<S::IO>(o.x * inv, o.y * inv), pack<S::IO>(o.z * inv, o.w * inv));
                *reinterpret_cast<uint2 *>(a.out + r * a.out_stride + ((int64_t)(head0 + q) * a.head_dim + d) * 2) = y;
            }
            if (q < heads && c < 2 && e4 == 0 && g == 0) write_lse<S>(a, r, head0 + q, top, l);
        } else {
            const Partial<S> p(to);
            __stcg(p.o + f * 32 + lane, o);
            if (c < 2 && e4 == 0 && g == 0) {
                __stcg(p.m + q, top);
                __stcg(p.l + q, l);
            }
        }
    }
}

// Offset, in 16-byte units, of the position `lane` of a tile in its buffer; kNoRow for a position that is left out.
template <int TOK>
__device__ __forceinline__ uint32_t row_offset(const AttendArgs &a, const Place<TOK> &p, bool report) {
    const int lane = threadIdx.x & 31;
    const int32_t pos = p.first / TOK * TOK + p.tile * TOK + lane;
    if (lane >= TOK || pos < p.first || pos >= p.len || p.r >= a.n_reqs) return kNoRow;
    const uint32_t col = (__umulhi((uint32_t)pos, a.block_mul) + (uint32_t)pos) >> a.block_shift;
    const int32_t blk = a.block_table[p.r * a.table_stride + col];
    if (blk < 0 || blk >= a.pool.n_blocks) {
        if (report && p.seg == 0) atomicAdd(a.pool.skipped, 1ull);
        return kNoRow;
    }
    return (uint32_t)blk * a.block_pitch16 + ((uint32_t)pos - col * (uint32_t)a.pool.block_size) * a.token_pitch16;
}

template <class S> __global__ void __launch_bounds__(kAttendThreads, S::CTAS) kvx_attend_planes(const __grid_constant__ AttendArgs a) {
    constexpr int TOK = S::TOK, NT = S::NT;
    extern __shared__ __align__(16) uint8_t smem[];                // [warp][2] partial results
    __shared__ int64_t s_seg[kAttendWarps][2];                     // first tile of each one's segment; -1: none
    __shared__ int32_t s_where[kAttendWarps][2][3];                // request, segment of the request, tiles
    __shared__ bool s_last;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int32_t group = a.n_q_heads / a.n_kv_heads, sets = (group + 8 * NT - 1) / (8 * NT), segs = a.n_kv_heads * sets;

    int32_t r0 = 0;
    int64_t before0 = 0;
    const Split split = split_batch<TOK>(a, segs, kAttendWarps, &r0, &before0);
    if ((int32_t)blockIdx.x >= split.ctas) return;
    const int64_t c_begin = split.begin(blockIdx.x), c_end = split.begin(blockIdx.x + 1);
    const int64_t x0 = c_begin + (c_end - c_begin) * w / kAttendWarps, x1 = c_begin + (c_end - c_begin) * (w + 1) / kAttendWarps;
    if (lane < 2) s_seg[w][lane] = -1;
    __syncwarp();

    if (x0 < x1) {
        uint32_t kr[S::SUB][S::KCH][2][4], vr[S::SUB][4][S::NP][S::PIECE / 4];
        uint32_t q[NT][S::KCH * S::KSTEP][2];
        float o[NT][S::NE / 2][4], m[NT][2], l[NT][2], sc[NT][2];
        Place<TOK> cur = locate<TOK>(a, segs, x0, r0, before0), nxt;
        const uint8_t *k_ptr, *v_ptr;                              // this lane's bytes of row 0 of the head

        auto pointers = [&](const Place<TOK> &p) {
            const int32_t kvh = p.seg / sets, shard = kvh / a.pool.heads_per_shard;
            const int64_t off = (int64_t)(kvh - shard * a.pool.heads_per_shard) * a.pool.head_pitch;
            k_ptr = a.pool.k[shard] + off + t * 16;
            v_ptr = a.pool.v[shard] + off + g * S::PIECE;
        };
        auto load_k = [&](uint32_t row) {
#pragma unroll
            for (int s = 0; s < S::SUB; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x = __shfl_sync(~0u, row, s * 16 + h * 8 + g);
                    const uint8_t *p = k_ptr + (uint64_t)x * 16;
#pragma unroll
                    for (int c = 0; c < S::KCH; ++c) load_row(kr[s][c][h], p + c * 64, x != kNoRow && c * 64 + t * 16 < a.head_dim * S::ESZ);
                }
        };
        auto load_v = [&](uint32_t row) {
#pragma unroll
            for (int s = 0; s < S::SUB; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {                      // positions 2t, 2t + 1, 2t + 8, 2t + 9
                    const uint32_t x = __shfl_sync(~0u, row, s * 16 + 2 * t + (j & 1) + (j >> 1) * 8);
                    const uint8_t *p = v_ptr + (uint64_t)x * 16;
#pragma unroll
                    for (int c = 0; c < S::NP; ++c)
                        load_row(vr[s][j][c], p + c * 8 * S::PIECE, x != kNoRow && c * 8 * S::PIECE + g * S::PIECE < a.head_dim * S::ESZ);
                }
        };
        // Queries of a segment. 8-bit caches multiply in f16: a bf16 row is brought by a power of two to where f16 holds
        // its elements exactly down to 2^-33 of the largest.
        auto load_q = [&](const Place<TOK> &p) {
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
                        if (qi < group && d < a.head_dim) x = __ldg(reinterpret_cast<const uint4 *>(src + d * 2));
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
                    const int e = top > 0.0f && top < INFINITY ? max(-100, min(100, 14 - ilogbf(top))) : 0;
                    const float up = __int_as_float((127 + e) << 23);
                    scale *= __int_as_float((127 - e) << 23);
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
        auto flush = [&](const Place<TOK> &p, int64_t from, int64_t to) {
            const int64_t begin = p.seg_begin(segs);
            const int32_t kvh = p.seg / sets, first = p.seg % sets * 8 * NT;
            const bool whole = from == begin && to == begin + p.tiles;
            const int slot = from == begin;
            if (!whole && lane == 0) {
                s_seg[w][slot] = begin;
                s_where[w][slot][0] = p.r;
                s_where[w][slot][1] = p.seg;
                s_where[w][slot][2] = p.tiles;
            }
            const Partial<S> part(smem + (w * 2 + slot) * S::PARTIAL);
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
                        const float inv = l[n][i] == 0.0f ? 0.0f : a.v_scale / l[n][i];
                        uint8_t *dst = a.out + p.r * a.out_stride + (int64_t)head * a.head_dim * 2;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int e = 0; e < S::NE / 2; e += 4) {
                                const int d = S::dim(g, h * (S::NE / 2) + e), c = 2 * h + i;
                                if (d < a.head_dim)
                                    *reinterpret_cast<uint2 *>(dst + d * 2) =
                                        make_uint2(pack<S::IO>(o[n][e][c] * inv, o[n][e + 1][c] * inv),
                                                   pack<S::IO>(o[n][e + 2][c] * inv, o[n][e + 3][c] * inv));
                            }
                        if (g == 0) write_lse<S>(a, p.r, head, m[n][i], l[n][i]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < S::NE / 2; e += 4)
                            part.o[((n * 4 + c) * (S::NE / 8) + e / 4) * 32 + lane] =
                                make_float4(o[n][e][c], o[n][e + 1][c], o[n][e + 2][c], o[n][e + 3][c]);
                    if (g == 0)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            part.m[n * 8 + 2 * t + i] = m[n][i];
                            part.l[n * 8 + 2 * t + i] = l[n][i];
                        }
                }
            }
        };

        uint32_t row = row_offset<TOK>(a, cur, true), row_next = kNoRow;
        pointers(cur);
        load_k(row);
        load_v(row);
        load_q(cur);
        int64_t from = x0;
        for (int64_t x = x0; x < x1; ++x) {
            nxt = cur;
            nxt.next(a, segs);
            const bool more = x + 1 < x1;
            row_next = more ? row_offset<TOK>(a, nxt, true) : kNoRow;

            float s[NT][S::SUB][4];
#pragma unroll
            for (int u = 0; u < S::SUB; ++u) {
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n][u][0] = s[n][u][1] = s[n][u][2] = s[n][u][3] = 0.0f;
#pragma unroll
                for (int c = 0; c < S::KCH; ++c) {
                    uint32_t (&k)[2][4] = kr[u][c];
#pragma unroll
                    for (int i = 0; i < S::KSTEP; ++i) {
                        uint32_t a0, a1, a2, a3;
                        if constexpr (S::F8) {
                            a0 = f16_of_codes(k[0][i]), a2 = f16_of_codes(k[0][i] >> 16);
                            a1 = f16_of_codes(k[1][i]), a3 = f16_of_codes(k[1][i] >> 16);
                        } else {
                            a0 = k[0][2 * i], a2 = k[0][2 * i + 1], a1 = k[1][2 * i], a3 = k[1][2 * i + 1];
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma<S::MT>(s[n][u], a0, a1, a2, a3, q[n][c * S::KSTEP + i][0], q[n][c * S::KSTEP + i][1]);
                    }
                }
            }
            if (more) {
                if (nxt.seg != cur.seg || nxt.r != cur.r) pointers(nxt);
                load_k(row_next);
            }
            uint32_t p_hi[NT][S::SUB][2], p_lo[NT][S::SUB][2];
#pragma unroll
            for (int u = 0; u < S::SUB; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool out = __shfl_sync(~0u, row, u * 16 + h * 8 + g) == kNoRow;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) s[n][u][2 * h + i] = out ? -INFINITY : s[n][u][2 * h + i] * sc[n][i];
                }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float old[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float top = m[n][i];
#pragma unroll
                    for (int u = 0; u < S::SUB; ++u) top = fmaxf(top, fmaxf(s[n][u][i], s[n][u][2 + i]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                    const float ref = top == -INFINITY ? 0.0f : top;
                    old[i] = fast_exp2(m[n][i] - ref);
                    m[n][i] = top;
                    l[n][i] *= old[i];
#pragma unroll
                    for (int u = 0; u < S::SUB; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float p = fast_exp2(s[n][u][2 * h + i] - ref);
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
                // Weights as a sum of two 16-bit values, so that their rounding does not add to that of the output;
                // one suffices for 8-bit caches with bf16 outputs, whose unit is 8 times that of the f16 weights.
#pragma unroll
                for (int u = 0; u < S::SUB; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float p0 = s[n][u][2 * h], p1 = s[n][u][2 * h + 1];
                        const uint32_t hi = pack<S::MT>(p0, p1);
                        p_hi[n][u][h] = transpose8x8(hi);
                        if constexpr (!(S::F8 && S::IO == KVX_BF16)) {
                            const float2 f = unpack<S::MT>(hi);
                            p_lo[n][u][h] = transpose8x8(pack<S::MT>(p0 - f.x, p1 - f.y));
                        }
                    }
            }
#pragma unroll
            for (int u = 0; u < S::SUB; ++u)
#pragma unroll
                for (int e = 0; e < S::NE / 2; ++e) {
                    uint32_t av[4];                                 // rows g (element e) and g + 8 (element e + NE / 2)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int el = e + (i & 1) * (S::NE / 2), j = (i >> 1) * 2;
                        const int c = el / S::PE, b = el % S::PE * S::ESZ;
                        const uint32_t x = vr[u][j][c][b / 4], y = vr[u][j + 1][c][b / 4];
                        if constexpr (S::F8) av[i] = f16_of_codes(__byte_perm(x, y, (b & 3) | ((b & 3) + 4) << 4));
                        else av[i] = __byte_perm(x, y, b & 2 ? 0x7632 : 0x5410);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma<S::MT>(o[n][e], av[0], av[1], av[2], av[3], p_hi[n][u][0], p_hi[n][u][1]);
                        if constexpr (!(S::F8 && S::IO == KVX_BF16))
                            mma<S::MT>(o[n][e], av[0], av[1], av[2], av[3], p_lo[n][u][0], p_lo[n][u][1]);
                    }
                }
            if (more) load_v(row_next);
            if (cur.tile + 1 == cur.tiles || !more) {
                flush(cur, from, x + 1);
                from = x + 1;
                if (more) load_q(nxt);
            }
            cur = nxt;
            row = row_next;
        }
    }
    __syncthreads();

    // Pieces of a segment that several warps of this CTA share, in order: the second of one warp, the first ones of those after it.
    uint8_t *const parts = a.scratch + kScratchCounters * sizeof(uint32_t);
    uint32_t *const arrived = (uint32_t *)a.scratch;
    for (int i = 0; i < 2 * kAttendWarps;) {
        const int64_t seg = s_seg[i >> 1][i & 1];
        if (seg < 0) {
            ++i;
            continue;
        }
        int ids[kAttendWarps + 1], n = 0, j = i;
        for (; j < 2 * kAttendWarps; ++j) {
            const int64_t other = s_seg[j >> 1][j & 1];
            if (other < 0) continue;
            if (other != seg) break;
            ids[n++] = j;
        }
        const int32_t r = s_where[i >> 1][i & 1][0], sg = s_where[i >> 1][i & 1][1], tiles = s_where[i >> 1][i & 1][2];
        const int32_t kvh = sg / sets, first = sg % sets * 8 * NT, head0 = kvh * group + first, heads = min(group - first, 8 * NT);
        const bool whole = seg >= c_begin && seg + tiles <= c_end;
        uint8_t *to = parts + (size_t)(blockIdx.x * 2 + (seg >= c_begin)) * S::PARTIAL;
        join<S, false>(a, n, [&](int x) { return smem + ids[x] * S::PARTIAL; }, whole, to, r, head0, heads);
        if (!whole) {
            const int32_t from = split.cta_of(seg), upto = split.cta_of(seg + tiles - 1);
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                s_last = atomicAdd(arrived + from, 1u) == (uint32_t)(upto - from);
                if (s_last) arrived[from] = 0;
                __threadfence();
            }
            __syncthreads();
            if (s_last)
                join<S, true>(a, upto - from + 1, [&](int x) { return parts + (size_t)((from + x) * 2 + (x == 0)) * S::PARTIAL; }, true, to, r,
                        head0, heads);
            __syncthreads();
        }
        i = j;
    }
}

// ------------------------------------------------------------------------------------------------

template <class S> static cudaError_t launch(const AttendArgs &a, int32_t sms, cudaStream_t stream) {
    constexpr int bytes = 2 * kAttendWarps * S::PARTIAL;
    static const cudaError_t set = cudaFuncSetAttribute(kvx_attend_planes<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (set != cudaSuccess) return set;
    kvx_attend_planes<S><<<S::CTAS * sms, kAttendThreads, bytes, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}

template <int VT, int IO> static cudaError_t launch(const AttendArgs &a, int32_t sms, cudaStream_t stream) {
    const bool wide = a.n_q_heads / a.n_kv_heads > 8;
    if (a.head_dim <= 64) return wide ? launch<Shape<VT, IO, 64, 2>>(a, sms, stream) : launch<Shape<VT, IO, 64, 1>>(a, sms, stream);
    if (a.head_dim <= 128) return wide ? launch<Shape<VT, IO, 128, 2>>(a, sms, stream) : launch<Shape<VT, IO, 128, 1>>(a, sms, stream);
    return launch<Shape<VT, IO, 256, 1>>(a, sms, stream);
}

// Counters of the segments that cross CTAs, then two partial results per CTA (at most two CTAs per SM).
size_t attend_scratch_bytes(int32_t sms) { return kScratchCounters * sizeof(uint32_t) + (size_t)4 * sms * kPartialMax; }

cudaError_t launch_attend(const AttendArgs &a, int32_t vt, int32_t io, int32_t sms, cudaStream_t stream) {
    if (a.latent) return launch_attend_latent(a, vt, io, sms, stream);
    if (vt == KVX_BF16) return launch<KVX_BF16, KVX_BF16>(a, sms, stream);
    if (vt == KVX_F16) return launch<KVX_F16, KVX_F16>(a, sms, stream);
    return io == KVX_BF16 ? launch<KVX_E4M3, KVX_BF16>(a, sms, stream) : launch<KVX_E4M3, KVX_F16>(a, sms, stream);
}

}  // namespace kvx
