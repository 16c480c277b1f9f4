// kvx_cache_attend over one plane of latents: keys of head_dim elements whose first v_dim are the values,
// all of a KV head's query heads (16 at a time) on the same rows.
//
// Per position 2 (head_dim + v_dim) flops for each query head meet head_dim bytes (or twice that): with 16
// query heads and 8-bit latents of 576 that is 60 flops a byte, more than the shared work of one warp can
// feed, and the output of 16 x 512 sums does not fit one warp's registers. So the 8 warps of a CTA take a
// tile of 64 (32) positions together:
//   scores   S^T = K Q^T: a warp takes half of the positions and a quarter of the elements, with its part
//            of the queries in registers; the quarters are summed through shared memory;
//   softmax  a warp takes two query heads; running maximum and sum stay in its registers;
//   values   O^T += V^T P^T: a warp takes 64 of the 512 elements, all positions.
// Rows come by bulk copies, two tiles deep. A row's pitch of 608 (1184) bytes, 96 (32) beyond a multiple of
// 128, keeps both kinds of reads off each other's banks: rows t = 0..3 of the values' reads fall on the four
// quarters of the banks, and the keys' reads take rows two apart. Two CTAs per SM fill each other's waits.
#include "kvx_attend.cuh"

#include <algorithm>

namespace kvx {

constexpr int kLatentWarps = 8, kLatentThreads = 32 * kLatentWarps, kLatentHeads = 16;
constexpr int kLatentFloat4 = kLatentHeads * kCacheMaxLatentValue / 4;                 // of a partial result
constexpr int kLatentPartial = kLatentFloat4 * 16 + 2 * kLatentHeads * 4;              // O, m, l
constexpr int kLatentMinTiles = 2;                                                     // of a CTA
constexpr uint64_t kLatentWaitNs = 2000000000ull;

template <int VT_, int IO_> struct LatentShape {
    static constexpr int VT = VT_, IO = IO_;
    static constexpr bool F8 = VT == KVX_E4M3;
    static constexpr int MT = F8 ? KVX_F16 : VT;
    static constexpr bool SPLIT = !(F8 && IO == KVX_BF16);        // weights in two 16-bit parts, as in kvx_attend_planes.cuh
    static constexpr int ESZ = F8 ? 1 : 2;
    static constexpr int TOK = F8 ? 64 : 32;
    static constexpr int KSTEP = F8 ? 4 : 2;                      // products per 64-byte chunk of a row
    static constexpr int CHUNKS = kCacheMaxLatent * ESZ / 64;     // 9 (18)
    static constexpr int CM = CHUNKS / 4;                         // of a quarter; 4 CM .. CHUNKS - 1 are left over
    static constexpr int MPW = TOK / 32;                          // 16-position products of half a tile
    static constexpr int PITCH = kCacheMaxLatent * ESZ + 32;
    static constexpr int STAGE = TOK * PITCH;
    static constexpr int SROW = TOK + 4;                          // floats of a head's scores in shared memory
    static constexpr int PENTRY = SPLIT ? 16 : 8;
    static constexpr int OFF_S = 2 * STAGE, OFF_P = OFF_S + 4 * kLatentHeads * SROW * 4;
    static constexpr int BYTES = OFF_P + TOK / 16 * 2 * 32 * PENTRY;
};

__device__ __forceinline__ uint32_t shared_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Waits for a phase of a stage's barrier, kLatentWaitNs at most.
__device__ __forceinline__ bool wait_full(uint64_t *bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t tries = 0;; ++tries) {
        uint32_t done;
        asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                     : "=r"(done) : "r"(shared_addr(bar)), "r"(parity) : "memory");
        if (done) return true;
        if ((tries & 63) == 0) {
            uint64_t now;
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
            if (!t0) t0 = now;
            else if (now - t0 > kLatentWaitNs) return false;
        }
    }
}

// What a CTA leaves for the joining kernel: the segment that begins in its stretch and goes on after it (pieces 0: none).
struct OpenSegment {
    int32_t r, seg, pieces, unused;
};

template <class S> __global__ void __launch_bounds__(kLatentThreads, 2) kvx_attend_latent(const __grid_constant__ AttendArgs a) {
    constexpr int TOK = S::TOK;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_full[2];
    __shared__ uint32_t s_live[2][2];                              // live positions of a stage's tile
    __shared__ float s_old[kLatentHeads], s_m[kLatentHeads], s_l[kLatentHeads], s_up[kLatentHeads];
    __shared__ int32_t s_timeout;
    float *const scores = (float *)(smem + S::OFF_S);
    uint8_t *const weights = smem + S::OFF_P;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int kq = w & 3, half = w >> 2;                           // quarter of the elements, half of the positions
    const int h = 2 * w + (lane >> 4), x = lane & 15;              // softmax: query head, place among its 16 lanes
    const int32_t group = a.n_q_heads / a.n_kv_heads, sets = (group + kLatentHeads - 1) / kLatentHeads, segs = a.n_kv_heads * sets;
    const uint32_t row_bytes = (uint32_t)a.head_dim * S::ESZ;

    wait_for_earlier();
    OpenSegment *const open = (OpenSegment *)a.scratch;
    uint8_t *const parts = a.scratch + kScratchCounters * sizeof(uint32_t);
    const Batch<TOK, kLatentWarps, kLatentMinTiles> batch(a, segs);
    if (threadIdx.x == 0) {
        if ((int32_t)blockIdx.x >= batch.split.ctas) open[blockIdx.x].pieces = 0;
        s_timeout = 0;
        for (int i = 0; i < 2; ++i) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_addr(&s_full[i])) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if ((int32_t)blockIdx.x >= batch.split.ctas) return;
    const int64_t c_begin = batch.split.begin(blockIdx.x), c_end = batch.split.begin(blockIdx.x + 1);
    const int32_t n_tiles = (int32_t)min(c_end - c_begin, (int64_t)INT32_MAX);
    if (a.head_dim < kCacheMaxLatent)                              // elements that no copy writes
        for (int i = threadIdx.x; i < 2 * S::STAGE / 16; i += kLatentThreads) *(uint4 *)(smem + i * 16) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();

    Place<TOK> cur = batch.locate(a, segs, c_begin), far = cur;

    // Warp 0: the block ids of tile `far`, and its rows' copies.
    int32_t blk[TOK / 32];
    uint32_t rest[TOK / 32];
    auto lookup = [&]() {
#pragma unroll
        for (int i = 0; i < TOK / 32; ++i) {
            const uint32_t pos = (uint32_t)far.first / TOK * TOK + (uint32_t)far.tile * TOK + i * 32 + lane;
            blk[i] = -2;
            if (pos < (uint32_t)far.first || pos >= (uint32_t)far.len) continue;
            const uint32_t col = (__umulhi(pos, a.block_mul) + pos) >> a.block_shift;
            blk[i] = max(a.block_table[far.r * a.table_stride + col], -1);
            rest[i] = (pos - col * (uint32_t)a.pool.block_size) * a.token_pitch16;
        }
    };
    auto copy_tile = [&](int stage) {
        const int32_t kvh = far.seg / sets, shard = kvh / a.pool.heads_per_shard;
        const uint8_t *base = a.pool.k[shard] + (int64_t)(kvh - shard * a.pool.heads_per_shard) * a.pool.head_pitch;
        uint8_t *const to = smem + stage * S::STAGE;
        const uint32_t bar = shared_addr(&s_full[stage]);
        uint32_t live[2] = {~0u, ~0u}, bytes = 0;
        bool dead = false;
#pragma unroll
        for (int i = 0; i < TOK / 32; ++i) {
            const bool in = blk[i] >= 0 && blk[i] < a.pool.n_blocks;
            if (!in && blk[i] != -2 && far.seg == 0) atomicAdd(a.pool.skipped, 1ull);
            live[i] = __ballot_sync(~0u, in);
            bytes += __popc(live[i]) * row_bytes;
            dead |= live[i] != ~0u;
        }
        if (dead) {                                                // rows that no copy fills read as zero
            for (int i = 0; i < TOK; ++i)
                if (!(live[i >> 5] >> (i & 31) & 1))
                    for (uint32_t b = lane * 16; b < row_bytes; b += 512) *(uint4 *)(to + i * S::PITCH + b) = make_uint4(0, 0, 0, 0);
        }
        if (lane < 2) s_live[stage][lane] = live[lane];
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
        __syncwarp();
#pragma unroll
        for (int i = 0; i < TOK / 32; ++i)
            if (live[i] >> lane & 1) {
                const uint8_t *src = base + ((uint64_t)((uint32_t)blk[i] * a.block_pitch16 + rest[i])) * 16;
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                 shared_addr(to + (i * 32 + lane) * S::PITCH)),
                             "l"(src), "r"(row_bytes), "r"(bar)
                             : "memory");
            }
    };
    if (w == 0) {
        lookup();
        copy_tile(0);
        far.next(a, segs);
        if (n_tiles > 1) {
            lookup();
            copy_tile(1);
            far.next(a, segs);
        }
        if (n_tiles > 2) lookup();
    }

    uint32_t q[S::CM + 1][S::KSTEP][2][2];                         // this quarter's chunks, then a left-over one
    float o[4][2][4], m = -INFINITY, l = 0.0f, scale = a.scale;    // m, l, scale: of head h
    const int left_chunk = 4 * S::CM + (S::F8 ? 0 : kq & 1);       // the left-over chunks go round the warps
    const bool left = (kq >> 1) == half;
    auto load_q = [&]() {
        const int32_t kvh = cur.seg / sets, first = cur.seg % sets * kLatentHeads;
        const uint8_t *src = a.q + cur.r * a.q_stride + (int64_t)(kvh * group + first) * a.head_dim * 2;
        if constexpr (S::F8 && S::IO == KVX_BF16) {                // a power of two per query, as in kvx_attend_planes.cuh
            float top = 0.0f;
            if (first + h < group)
                for (int d = x * 8; d < a.head_dim; d += 128) {
                    const uint4 y = __ldg(reinterpret_cast<const uint4 *>(src + ((int64_t)h * a.head_dim + d) * 2));
                    for (uint32_t z : {y.x, y.y, y.z, y.w}) {
                        const float2 f = unpack<KVX_BF16>(z);
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            const int e = top > 0.0f && top < INFINITY ? max(-100, min(100, 14 - ilogbf(top))) : 0;
            scale = a.scale * __int_as_float((127 - e) << 23);
            if (x == 0) s_up[h] = __int_as_float((127 + e) << 23);
            __syncthreads();
        }
#pragma unroll
        for (int c = 0; c <= S::CM; ++c)
#pragma unroll
            for (int k = 0; k < S::KSTEP / 2; ++k)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int chunk = c < S::CM ? kq * S::CM + c : left_chunk, d = (chunk * 64 + t * 16) / S::ESZ + k * 8;
                    uint4 y = make_uint4(0, 0, 0, 0);
                    if (first + n * 8 + g < group && d < a.head_dim)
                        y = __ldg(reinterpret_cast<const uint4 *>(src + ((int64_t)(n * 8 + g) * a.head_dim + d) * 2));
                    uint32_t z[4] = {y.x, y.y, y.z, y.w};
                    if constexpr (S::F8 && S::IO == KVX_BF16) {
                        const float up = s_up[n * 8 + g];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 f = unpack<KVX_BF16>(z[i]);
                            z[i] = pack<KVX_F16>(f.x * up, f.y * up);
                        }
                    }
                    q[c][2 * k][n][0] = z[0];
                    q[c][2 * k][n][1] = z[1];
                    q[c][2 * k + 1][n][0] = z[2];
                    q[c][2 * k + 1][n][1] = z[3];
                }
        m = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int n = 0; n < 2; ++n) o[e][n][0] = o[e][n][1] = o[e][n][2] = o[e][n][3] = 0.0f;
    };
    load_q();

    bool begun = cur.seg_begin(segs) == c_begin;                   // the segment at hand begins in this CTA
    int32_t last_r = 0, last_seg = 0, last_pieces = 0;
    for (int32_t k = 0; k < n_tiles; ++k) {
        const int stage = k & 1;
        const uint32_t rows = shared_addr(smem + stage * S::STAGE);
        if (!wait_full(&s_full[stage], k >> 1 & 1)) s_timeout = 1;

        // scores: rows g and g + 8 of a product are positions whose low two bits are swapped
        float s[S::MPW][2][4];
        const uint32_t my_row = rows + (half * S::MPW * 16 + ((g & 4) | (g & 1) << 1 | (g >> 1 & 1))) * S::PITCH + t * 16;
        auto score_chunk = [&](int i, int c, int chunk) {
            uint32_t ka[2][4];
            shared_read(ka[0], my_row + i * 16 * S::PITCH + chunk * 64);
            shared_read(ka[1], my_row + (i * 16 + 8) * S::PITCH + chunk * 64);
#pragma unroll
            for (int y = 0; y < S::KSTEP; ++y) {
                uint32_t a0, a1, a2, a3;
                if constexpr (S::F8) {
                    a0 = f16_of_codes(ka[0][y]), a2 = f16_of_codes(ka[0][y] >> 16);
                    a1 = f16_of_codes(ka[1][y]), a3 = f16_of_codes(ka[1][y] >> 16);
                } else {
                    a0 = ka[0][2 * y], a2 = ka[0][2 * y + 1], a1 = ka[1][2 * y], a3 = ka[1][2 * y + 1];
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) mma<S::MT>(s[i][n], a0, a1, a2, a3, q[c][y][n][0], q[c][y][n][1]);
            }
        };
#pragma unroll
        for (int i = 0; i < S::MPW; ++i) {
#pragma unroll
            for (int n = 0; n < 2; ++n) s[i][n][0] = s[i][n][1] = s[i][n][2] = s[i][n][3] = 0.0f;
#pragma unroll
            for (int c = 0; c < S::CM; ++c) score_chunk(i, c, kq * S::CM + c);
            if (left && (S::MPW == 1 || i == (kq & 1))) score_chunk(i, S::CM, left_chunk);
        }
        // [quarter][head][16-position product][position % 4][position / 4]
#pragma unroll
        for (int i = 0; i < S::MPW; ++i)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int pos = ((g & 4) | (g & 1) << 1 | (g >> 1 & 1)) + (c >> 1) * 8;
                    scores[(kq * kLatentHeads + n * 8 + 2 * t + (c & 1)) * S::SROW + (half * S::MPW + i) * 16 + (pos & 3) * 4 + (pos >> 2)] = s[i][n][c];
                }
        __syncthreads();
        if (s_timeout) {
            if (k + 1 < n_tiles) wait_full(&s_full[stage ^ 1], k + 1 >> 1 & 1);   // its copies may be under way
            break;
        }

        // softmax of head h: lane x has positions 16 u + y + 4 j for (u, y) = (x / 4, x % 4) and all j, or (x / 8, x / 2 % 4) and two j
        {
            constexpr int E = TOK / 16;
            float p[E];
#pragma unroll
            for (int e = 0; e < E; ++e) p[e] = 0.0f;
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) {
                const float *src = scores + (k4 * kLatentHeads + h) * S::SROW + x * E;
                if constexpr (E == 4) {
                    const float4 y = *(const float4 *)src;
                    p[0] += y.x, p[1] += y.y, p[2] += y.z, p[3] += y.w;
                } else {
                    const float2 y = *(const float2 *)src;
                    p[0] += y.x, p[1] += y.y;
                }
            }
            const int u = E == 4 ? x >> 2 : x >> 3, y = E == 4 ? x & 3 : x >> 1 & 3, j0 = E == 4 ? 0 : 2 * (x & 1);
            if ((s_live[stage][0] & s_live[stage][1]) != ~0u)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int pos = 16 * u + y + 4 * (j0 + e);
                    if (!(s_live[stage][pos >> 5] >> (pos & 31) & 1)) p[e] = -INFINITY;
                }
            float top = p[0];
#pragma unroll
            for (int e = 1; e < E; ++e) top = fmaxf(top, p[e]);
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            top = fmaxf(m, top * scale);
            const float ref = top == -INFINITY ? 0.0f : top, old = fast_exp2(m - ref);
            m = top;
            l *= old;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                p[e] = fast_exp2(fmaf(p[e], scale, -ref));
                l += p[e];
            }
            if (x == 0) s_old[h] = old;
            uint8_t *to = weights + ((u * 2 + (h >> 3)) * 32 + (h & 7) * 4 + y) * S::PENTRY + j0 * 2;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const uint32_t hi = pack<S::MT>(p[e], p[e + 1]);
                *(uint32_t *)(to + e * 2) = hi;
                if constexpr (S::SPLIT) {
                    const float2 f = unpack<S::MT>(hi);
                    *(uint32_t *)(to + 8 + e * 2) = pack<S::MT>(p[e] - f.x, p[e + 1] - f.y);
                }
            }
        }
        __syncthreads();

        // values: k elements (2t, 2t + 1, 2t + 8, 2t + 9) of a product are positions t, t + 4, t + 8, t + 12
        {
            float old[2][2];
            bool moved = false;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    old[n][i] = s_old[n * 8 + 2 * t + i];
                    moved |= old[n][i] != 1.0f;
                }
            if (__any_sync(~0u, moved)) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        o[e][n][0] *= old[n][0];
                        o[e][n][1] *= old[n][1];
                        o[e][n][2] *= old[n][0];
                        o[e][n][3] *= old[n][1];
                    }
            }
            const uint32_t my_values = rows + t * S::PITCH + (w * 64 + g * 8) * S::ESZ, my_weights = shared_addr(weights) + lane * S::PENTRY;
#pragma unroll
            for (int u = 0; u < TOK / 16; ++u) {
                uint32_t v[4][S::ESZ * 2], p[2][S::PENTRY / 4];
#pragma unroll
                for (int n = 0; n < 2; ++n) shared_read(p[n], my_weights + (u * 2 + n) * 32 * S::PENTRY);
#pragma unroll
                for (int j = 0; j < 4; ++j) shared_read(v[j], my_values + (u * 16 + j * 4) * S::PITCH);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t av[4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if constexpr (S::F8) {
                            const uint32_t z = __byte_perm(v[2 * j][e / 2], v[2 * j + 1][e / 2], e & 1 ? 0x7362 : 0x5140);
                            av[2 * j] = f16_of_codes(z);
                            av[2 * j + 1] = f16_of_codes(z >> 16);
                        } else {
                            av[2 * j] = __byte_perm(v[2 * j][e], v[2 * j + 1][e], 0x5410);
                            av[2 * j + 1] = __byte_perm(v[2 * j][e], v[2 * j + 1][e], 0x7632);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma<S::MT>(o[e][n], av[0], av[1], av[2], av[3], p[n][0], p[n][1]);
                        if constexpr (S::SPLIT) mma<S::MT>(o[e][n], av[0], av[1], av[2], av[3], p[n][2], p[n][3]);
                    }
                }
            }
        }

        const bool ends = cur.tile + 1 == cur.tiles;
        if (ends || k + 1 == n_tiles) {
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) l += __shfl_xor_sync(~0u, l, d);
            if (x == 0) {
                s_m[h] = m;
                s_l[h] = l;
            }
            __syncthreads();
            const int32_t kvh = cur.seg / sets, first = cur.seg % sets * kLatentHeads, head0 = kvh * group + first;
            const int32_t heads = min(group - first, kLatentHeads);
            if (ends && begun) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int qh = n * 8 + 2 * t + i, d = w * 64 + g * 8;
                        if (qh >= heads || d >= a.v_dim) continue;
                        const float inv = s_l[qh] == 0.0f ? 0.0f : a.v_scale / s_l[qh];
                        uint4 y;
                        y.x = pack<S::IO>(o[0][n][i] * inv, o[0][n][2 + i] * inv);
                        y.y = pack<S::IO>(o[1][n][i] * inv, o[1][n][2 + i] * inv);
                        y.z = pack<S::IO>(o[2][n][i] * inv, o[2][n][2 + i] * inv);
                        y.w = pack<S::IO>(o[3][n][i] * inv, o[3][n][2 + i] * inv);
                        *reinterpret_cast<uint4 *>(a.out + cur.r * a.out_stride + ((int64_t)(head0 + qh) * a.v_dim + d) * 2) = y;
                    }
                if (a.lse && threadIdx.x < heads)
                    a.lse[(int64_t)cur.r * a.n_q_heads + head0 + threadIdx.x] =
                        s_l[threadIdx.x] == 0.0f ? -INFINITY : (s_m[threadIdx.x] + log2f(s_l[threadIdx.x])) * kLn2;
            } else {
                uint8_t *const part = parts + (size_t)(blockIdx.x * 2 + begun) * kLatentPartial;
                float4 *const po = (float4 *)part;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            __stcg(po + (((w * 2 + n) * 2 + i) * 2 + e) * 32 + lane,
                                   make_float4(o[2 * e][n][i], o[2 * e][n][2 + i], o[2 * e + 1][n][i], o[2 * e + 1][n][2 + i]));
                if (threadIdx.x < kLatentHeads) {
                    float *const ml = (float *)(part + kLatentFloat4 * 16);
                    __stcg(ml + threadIdx.x, s_m[threadIdx.x]);
                    __stcg(ml + kLatentHeads + threadIdx.x, s_l[threadIdx.x]);
                }
                if (begun) {
                    last_r = cur.r;
                    last_seg = cur.seg;
                    last_pieces = batch.split.cta_of(cur.seg_begin(segs) + cur.tiles - 1) - blockIdx.x + 1;
                }
            }
        }
        if (k + 1 < n_tiles) {
            cur.next(a, segs);
            __syncthreads();                                       // nobody reads this stage any more
            if (w == 0 && k + 2 < n_tiles) {
                copy_tile(stage);
                far.next(a, segs);
                if (k + 3 < n_tiles) lookup();
            }
            if (ends) {
                begun = true;
                load_q();
            }
        }
    }
    if (s_timeout && threadIdx.x == 0) atomicAdd(a.pool.skipped + 1, 1ull);
    if (threadIdx.x == 0) open[blockIdx.x] = OpenSegment{last_r, last_seg, s_timeout ? 0 : last_pieces, 0};
}

// Joins the segments that go over several CTAs: 64 value elements of one segment at a time, 256 threads for its float4s four
// times over, each with every fourth piece.
constexpr int kJoinThreads = 1024, kJoinGroups = kJoinThreads / 256, kJoinPieces = 256;

template <int IO> __global__ void __launch_bounds__(kJoinThreads, 1) kvx_attend_latent_join(const __grid_constant__ AttendArgs a, int ctas) {
    __shared__ int32_t s_list[kJoinThreads], s_count[kJoinThreads / 32], s_n;
    __shared__ float s_w[kJoinPieces][kLatentHeads];           // weights of 256 pieces at a time
    __shared__ float4 s_o[kJoinGroups - 1][256];
    __shared__ float s_l[kLatentHeads], s_m[kLatentHeads];
    wait_for_earlier();
    const OpenSegment *const open = (const OpenSegment *)a.scratch;
    const uint8_t *const parts = a.scratch + kScratchCounters * sizeof(uint32_t);
    const int32_t group = a.n_q_heads / a.n_kv_heads, sets = (group + kLatentHeads - 1) / kLatentHeads;
    {                                                              // in order: every CTA has to number them alike
        const uint32_t found = __ballot_sync(~0u, (int)threadIdx.x < ctas && open[threadIdx.x].pieces > 0);
        if ((threadIdx.x & 31) == 0) s_count[threadIdx.x >> 5] = __popc(found);
        __syncthreads();
        int before = 0;
        for (int i = 0; i < (int)(threadIdx.x >> 5); ++i) before += s_count[i];
        if (found >> (threadIdx.x & 31) & 1) s_list[before + __popc(found & ((1u << (threadIdx.x & 31)) - 1))] = threadIdx.x;
        if (threadIdx.x == kJoinThreads - 1) s_n = before + __popc(found);
        __syncthreads();
    }
    for (int item = blockIdx.x; item < s_n * kLatentWarps; item += gridDim.x) {
        const int cta = s_list[item / kLatentWarps], w = item % kLatentWarps;
        const OpenSegment seg = open[cta];
        auto part = [&](int x) { return parts + (size_t)((cta + x) * 2 + (x == 0)) * kLatentPartial; };
        auto ml = [&](int x) { return (const float *)(part(x) + kLatentFloat4 * 16); };
        const int f = threadIdx.x & 255, piece0 = threadIdx.x >> 8;
        const int n = f >> 7, i = f >> 6 & 1, e4 = f >> 5 & 1, lane = f & 31, t = lane & 3, g = lane >> 2, q = n * 8 + 2 * t + i;
        // maxima and sums: head threadIdx / 64, 64 threads each
        {
            const int hq = threadIdx.x >> 6, y = threadIdx.x & 63;
            float top = -INFINITY, l = 0.0f;
            for (int x = y; x < seg.pieces; x += 64) top = fmaxf(top, __ldcg(ml(x) + hq));
            __syncthreads();
            float *const red = &s_w[0][0];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
            __syncthreads();
            top = fmaxf(red[hq * 2], red[hq * 2 + 1]);
            const float ref = top == -INFINITY ? 0.0f : top;
            for (int x = y; x < seg.pieces; x += 64) l += fast_exp2(__ldcg(ml(x) + hq) - ref) * __ldcg(ml(x) + kLatentHeads + hq);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) l += __shfl_xor_sync(~0u, l, d);
            __syncthreads();
            if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = l;
            __syncthreads();
            if (y == 0) {
                s_m[hq] = top;
                s_l[hq] = red[hq * 2] + red[hq * 2 + 1];
            }
        }
        float4 o = make_float4(0, 0, 0, 0);
        for (int x0 = 0; x0 < seg.pieces; x0 += kJoinPieces) {
            const int here = min(seg.pieces - x0, kJoinPieces);
            __syncthreads();
            for (int y = threadIdx.x; y < here * kLatentHeads; y += kJoinThreads) {
                const float top = s_m[y % kLatentHeads];
                s_w[y / kLatentHeads][y % kLatentHeads] = fast_exp2(__ldcg(ml(x0 + y / kLatentHeads) + y % kLatentHeads) - (top == -INFINITY ? 0.0f : top));
            }
            __syncthreads();
#pragma unroll 8
            for (int x = piece0; x < here; x += kJoinGroups) {
                const float4 y = __ldcg((const float4 *)part(x0 + x) + w * 256 + f);
                const float z = s_w[x][q];
                o.x += z * y.x;
                o.y += z * y.y;
                o.z += z * y.z;
                o.w += z * y.w;
            }
        }
        if (piece0) s_o[piece0 - 1][f] = o;
        __syncthreads();
        if (piece0 == 0) {
#pragma unroll
            for (int x = 0; x < kJoinGroups - 1; ++x) {
                const float4 y = s_o[x][f];
                o = make_float4(o.x + y.x, o.y + y.y, o.z + y.z, o.w + y.w);
            }
            const int32_t first = seg.seg % sets * kLatentHeads, head = seg.seg / sets * group + first + q, d = w * 64 + g * 8 + e4 * 4;
            if (first + q < group) {
                const float l = s_l[q], inv = l == 0.0f ? 0.0f : a.v_scale / l;
                if (d < a.v_dim)
                    *reinterpret_cast<uint2 *>(a.out + seg.r * a.out_stride + ((int64_t)head * a.v_dim + d) * 2) =
                        make_uint2(pack<IO>(o.x * inv, o.y * inv), pack<IO>(o.z * inv, o.w * inv));
                if (a.lse && w == 0 && e4 == 0 && g == 0)
                    a.lse[(int64_t)seg.r * a.n_q_heads + head] = l == 0.0f ? -INFINITY : (s_m[q] + log2f(l)) * kLn2;
            }
        }
        __syncthreads();
    }
}

size_t latent_scratch_bytes(int32_t sms) { return kScratchCounters * sizeof(uint32_t) + (size_t)4 * sms * kLatentPartial; }

template <class S> static cudaError_t launch(const AttendArgs &a, int32_t sms, cudaStream_t stream) {
    static const cudaError_t set = cudaFuncSetAttribute(kvx_attend_latent<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
    if (set != cudaSuccess) return set;
    const cudaError_t e = launch_after(kvx_attend_latent<S>, dim3(2 * sms), kLatentThreads, S::BYTES, stream, a);
    return e != cudaSuccess ? e : launch_after(kvx_attend_latent_join<S::IO>, dim3(sms), kJoinThreads, 0, stream, a, 2 * sms);
}

cudaError_t launch_attend_latent(const AttendArgs &a, int32_t vt, int32_t io, int32_t sms, cudaStream_t stream) {
    if (vt == KVX_BF16) return launch<LatentShape<KVX_BF16, KVX_BF16>>(a, sms, stream);
    if (vt == KVX_F16) return launch<LatentShape<KVX_F16, KVX_F16>>(a, sms, stream);
    return io == KVX_BF16 ? launch<LatentShape<KVX_E4M3, KVX_BF16>>(a, sms, stream) : launch<LatentShape<KVX_E4M3, KVX_F16>>(a, sms, stream);
}

}  // namespace kvx
