// kvx_cache_attend over one plane of latents: keys of head_dim elements whose first v_dim are the values,
// all of a KV head's query heads (16 at a time) on the same rows. Here those that the tensor maps of
// kvx_latent_tensor.cu cannot describe (several shards, heads with a gap); and the kernel that joins the
// parts of both.
//
// Per position 2 (head_dim + v_dim) flops for each query head meet 2 head_dim bytes: 30 flops a byte with 16
// query heads, more than the shared work of one warp can feed, and the output of 16 x 512 sums does not fit
// one warp's registers. So the 8 warps of a CTA take a tile of 32 positions (64 of 8 bits) together:
//   scores   S^T = K Q^T: a warp takes half of the positions and a quarter of the elements, with its part
//            of the queries in registers; the quarters are summed through shared memory;
//   softmax  a warp takes two query heads; running maximum and sum stay in its registers;
//   values   O^T += V^T P^T: a warp takes 64 of the 512 elements, all positions.
// Rows come by bulk copies, two tiles deep, a warp's share each (one warp for all of them was late at every
// barrier: 293 us where this takes 212). A row's pitch of 1184 (608) bytes, 32 (96) beyond a multiple of
// 128, keeps both kinds of reads off each other's banks: rows t = 0..3 of the values' reads fall on the four
// quarters of the banks, and the keys' reads take rows two apart. Two CTAs per SM fill each other's waits.
//
// Measured with 16 query heads: 64 requests of 8000 bf16 latents of 576 144 us, 4.1 TB/s, and 64 sessions of
// 2048 to 32768 8-bit ones 258 us (212 with weights as one f16 value), where the tcgen05 kernel takes 108 and 116. Bound
// by instruction issue (1.9 a clock, 95 warp instructions a position), with 78 to 142 bytes a thread spilled. Scores by 8-bit warp products (mma.sync e4m3, queries as two
// codes) were exact enough but took 395 us: the form costs ten instructions on sm_103a.
#include "kvx_latent.cuh"

namespace kvx {

constexpr int kLatentWarps = 8, kLatentThreads = 32 * kLatentWarps;
constexpr int kLatentMinTiles = 2;                                                     // of a CTA

template <int VT_, int IO_> struct LatentShape {
    static constexpr int VT = VT_, IO = IO_;
    static constexpr bool F8 = VT == KVX_E4M3;
    static constexpr int MT = F8 ? KVX_F16 : VT;
    // A weight is the sum of two 16-bit values: 2^-17 of it is left, f16: 2^-23. f16 weights are taken times 2^15, as in
    // kvx_attend_planes.cuh, so that those of 2^-39 of the largest still count. (An infinite value is an infinite key too, so
    // its weight is NaN or 0 by the definition, and the parts' signs do not matter here.)
    static constexpr float UP = MT == KVX_F16 ? 15.0f : 0.0f;
    static constexpr int ESZ = F8 ? 1 : 2;
    static constexpr int TOK = F8 ? 64 : 32;
    static constexpr int KSTEP = F8 ? 4 : 2;                      // products per 64-byte chunk of a row
    static constexpr int CHUNKS = kCacheMaxLatent * ESZ / 64;     // 9 (18)
    static constexpr int CM = CHUNKS / 4;                         // of a quarter; 4 CM .. CHUNKS - 1 are left over
    static constexpr int MPW = TOK / 32;                          // 16-position products of half a tile
    static constexpr int PITCH = kCacheMaxLatent * ESZ + 32;
    static constexpr int STAGE = TOK * PITCH;
    static constexpr int ROWS = TOK / kLatentWarps;               // copied by a warp
    static constexpr int PENTRY = 16;
    static constexpr int OFF_S = 2 * STAGE, OFF_P = OFF_S + 4 * kLatentHeads * TOK * 4;
    static constexpr int BYTES = OFF_P + TOK / 16 * 2 * 32 * PENTRY;
};

// Position s of the four that an entry of the weights holds, from the first.
__device__ __forceinline__ int entry_position(int s) { return 4 * ((s & 1) * 2 + (s >> 1)); }

template <class S> __global__ void __launch_bounds__(kLatentThreads, 2) kvx_attend_latent(const __grid_constant__ AttendArgs a) {
    constexpr int TOK = S::TOK;
    using Line = Place<TOK, 0>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_full[2], s_never;
    __shared__ __align__(8) uint8_t s_live[2][kLatentWarps];       // live positions of a stage's tile, a warp's rows each
    __shared__ Line s_cur, s_far;                            // this tile, and the next one to look up
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
    const Batch<TOK, kLatentWarps, kLatentMinTiles, 0, 0> batch(a, segs);
    if (threadIdx.x == 0) {
        if ((int32_t)blockIdx.x >= batch.split.ctas) open[blockIdx.x].pieces = 0;
        s_timeout = 0;
        for (int i = 0; i < 2; ++i) asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_addr(&s_full[i])), "n"(kLatentWarps) : "memory");
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_addr(&s_never)) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if ((int32_t)blockIdx.x >= batch.split.ctas) return;
    const int64_t c_begin = batch.split.begin(blockIdx.x), c_end = batch.split.begin(blockIdx.x + 1);
    const int32_t n_tiles = (int32_t)min(c_end - c_begin, (int64_t)INT32_MAX);
    if (a.head_dim < kCacheMaxLatent)                              // elements that no copy writes
        for (int i = threadIdx.x; i < 2 * S::STAGE / 16; i += kLatentThreads) *(uint4 *)(smem + i * 16) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();

    {
        int64_t x = c_begin;
        const Line begin = batch.locate(a, segs, x);
        if (threadIdx.x == 0) s_cur = s_far = begin;
    }
    __syncthreads();

    // A warp copies ROWS rows of each tile: the block id of lane x's row, its place in the block, and where its head begins.
    // A row that is not live (blk -2: no such position) is filled with zeros.
    int32_t blk = -2;
    uint32_t rest = 0;
    const uint8_t *base = nullptr;
    bool report = false;
    auto lookup = [&]() {
        const int32_t seg = s_far.seg, first = s_far.first, kvh = seg / sets, shard = kvh / a.pool.heads_per_shard;
        const uint32_t pos = (uint32_t)first / TOK * TOK + (uint32_t)s_far.tile * TOK + w * S::ROWS + lane;
        base = a.pool.k[shard] + (int64_t)(kvh - shard * a.pool.heads_per_shard) * a.pool.head_pitch;
        report = seg == 0;
        blk = -2;
        if (lane >= S::ROWS || pos < (uint32_t)first || pos >= (uint32_t)s_far.len) return;
        const uint32_t col = (__umulhi(pos, a.block_mul) + pos) >> a.block_shift;
        blk = max(a.block_table[s_far.r * a.table_stride + col], -1);
        rest = (pos - col * (uint32_t)a.pool.block_size) * a.token_pitch16;
    };
    auto copy_rows = [&](int stage) {
        uint8_t *const to = smem + stage * S::STAGE + w * S::ROWS * S::PITCH;
        const uint32_t bar = shared_addr(&s_full[stage]);
        const bool in = blk >= 0 && blk < a.pool.n_blocks;
        if (!in && blk != -2 && report) atomicAdd(a.pool.skipped, 1ull);
        const uint32_t live = __ballot_sync(~0u, in);
        if (live != (1u << S::ROWS) - 1)
            for (int i = 0; i < S::ROWS; ++i)
                if (!(live >> i & 1))
                    for (uint32_t b = lane * 16; b < row_bytes; b += 512) *(uint4 *)(to + i * S::PITCH + b) = make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            s_live[stage][w] = (uint8_t)live;
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(__popc(live) * row_bytes) : "memory");
        }
        __syncwarp();
        if (in)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             shared_addr(to + lane * S::PITCH)),
                         "l"(base + (uint64_t)((uint32_t)blk * a.block_pitch16 + rest) * 16), "r"(row_bytes), "r"(bar)
                         : "memory");
    };
    // Thread 0 moves s_far on where a barrier stands before and after.
    auto advance = [&](Line &p) {
        int64_t x = 0;
        if (threadIdx.x == 0) p.next(a, segs, x);
    };
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < n_tiles) {
            lookup();
            if (k < 2) copy_rows(k);
            __syncthreads();
            if (k + 1 < n_tiles) advance(s_far);
            __syncthreads();
        }

    uint32_t q[S::CM + 1][S::KSTEP][2][2];                         // this quarter's chunks, then a left-over one
    float o[4][2][4], m = -INFINITY, l = 0.0f, scale = a.scale;    // m, l, scale: of head h
    const int left_chunk = 4 * S::CM + (S::F8 ? 0 : kq & 1);       // the left-over chunks go round the warps
    const bool left = (kq >> 1) == half;
    auto load_q = [&]() {
        const int32_t kvh = s_cur.seg / sets, first = s_cur.seg % sets * kLatentHeads;
        const uint8_t *src = a.q + s_cur.r * a.q_stride + (int64_t)(kvh * group + first) * a.head_dim * 2;
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
            const int e = top > 0.0f && top < INFINITY ? max(-126, min(100, 14 - ilogbf(top))) : 0;
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

    bool begun = s_cur.seg_begin(segs) == c_begin;                 // the segment at hand begins in this CTA
    int32_t tiles_left = s_cur.tiles - s_cur.tile;                 // of it
    OpenSegment opened = {0, 0, 0, 0};
    for (int32_t k = 0; k < n_tiles; ++k) {
        const int stage = k & 1;
        const uint32_t rows = shared_addr(smem + stage * S::STAGE);
        if (!wait_full(a.stall && blockIdx.x == 0 ? &s_never : &s_full[stage], a.stall && blockIdx.x == 0 ? 0 : k >> 1 & 1, a.wait_ns)) s_timeout = 1;

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
                    f16_of_codes(ka[0][y], a0, a2);
                    f16_of_codes(ka[1][y], a1, a3);
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
        // [quarter][head][16-position product][position % 4][place in the entry], swizzled by the head for the two stores of a lane
#pragma unroll
        for (int i = 0; i < S::MPW; ++i)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int word = (half * S::MPW + i) * 16 + ((g & 1) << 1 | (g >> 1 & 1)) * 4 + (g >> 2) * 2;
                    *(float2 *)(scores + (kq * kLatentHeads + n * 8 + 2 * t + c) * TOK + (word ^ (t & 1) * 16 ^ (t >> 1) * 2)) =
                        make_float2(s[i][n][c], s[i][n][2 + c]);
                }
        __syncthreads();
        if (s_timeout) {
            for (int i = 0; i < 2; ++i)                            // no copy outlives the CTA: this tile's, and the next one's
                if (k + i < n_tiles) wait_full(&s_full[stage ^ i], k + i >> 1 & 1, kCacheWaitNs);
            break;
        }
        if (k > 0 && k + 3 < n_tiles) advance(s_far);

        // softmax of head h: lane x has an entry (or half of one) of the weights: positions 16 u + y + entry_position(s)
        {
            constexpr int E = TOK / 16;
            const int u = E == 4 ? x >> 2 : x >> 3, y = E == 4 ? x & 3 : x >> 1 & 3, s0 = E == 4 ? 0 : 2 * (x & 1), th = h >> 1 & 3;
            const float *src = scores + h * TOK + (u * 16 + y * 4 + s0 ^ (th & 1) * 16 ^ (E == 4 ? 0 : (th >> 1) * 2));
            float p[E];
#pragma unroll
            for (int e = 0; e < E; ++e) p[e] = 0.0f;
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4, src += kLatentHeads * TOK) {
                if constexpr (E == 4) {
                    const float4 z = *(const float4 *)src;
                    p[0] += z.x, p[1] += z.y, p[2] += z.z, p[3] += z.w;
                } else {
                    const float2 z = *(const float2 *)src;
                    p[0] += z.x, p[1] += z.y;
                }
            }
            if (E == 4 && th >> 1) {
                const float z0 = p[0], z1 = p[1];
                p[0] = p[E - 2], p[1] = p[E - 1], p[E - 2] = z0, p[E - 1] = z1;
            }
            const uint64_t live = *(const uint64_t *)s_live[stage];
            if (live != (S::ROWS == 8 ? ~0ull : 0x0f0f0f0f0f0f0f0full))
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int pos = 16 * u + y + entry_position(s0 + e);
                    if (!(live >> (pos / S::ROWS * 8 + pos % S::ROWS) & 1)) p[e] = -INFINITY;
                }
            float top = p[0];
#pragma unroll
            for (int e = 1; e < E; ++e) top = fmaxf(top, p[e]);
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            top = fmaxf(m, fmaf(top, scale, -S::UP));
            const float ref = top == -INFINITY ? 0.0f : top, old = fast_exp2(m - ref);
            m = top;
            l *= old;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                p[e] = fast_exp2(fmaf(p[e], scale, -ref));
                l += p[e];
            }
            if (x == 0) s_old[h] = old;
            uint8_t *to = weights + ((u * 2 + (h >> 3)) * 32 + (h & 7) * 4 + y) * S::PENTRY + s0 * 2;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const uint32_t hi = pack<S::MT>(p[e], p[e + 1]);
                *(uint32_t *)(to + e * 2) = hi;
                const float2 f = unpack<S::MT>(hi);
                *(uint32_t *)(to + 8 + e * 2) = pack<S::MT>(p[e] - f.x, p[e + 1] - f.y);
            }
        }
        __syncthreads();

        // values: k elements (2t, 2t + 1, 2t + 8, 2t + 9) of a product are the positions of an entry
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
                for (int j = 0; j < 4; ++j) shared_read(v[j], my_values + (u * 16 + entry_position(j)) * S::PITCH);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t av[4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if constexpr (S::F8) {
                            const uint32_t z = __byte_perm(v[2 * j][e / 2], v[2 * j + 1][e / 2], e & 1 ? 0x7362 : 0x5140);
                            f16_of_codes(z, av[2 * j], av[2 * j + 1]);
                        } else {
                            av[2 * j] = __byte_perm(v[2 * j][e], v[2 * j + 1][e], 0x5410);
                            av[2 * j + 1] = __byte_perm(v[2 * j][e], v[2 * j + 1][e], 0x7632);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma<S::MT>(o[e][n], av[0], av[1], av[2], av[3], p[n][0], p[n][1]);
                        mma<S::MT>(o[e][n], av[0], av[1], av[2], av[3], p[n][2], p[n][3]);
                    }
                }
            }
        }

        const bool ends = --tiles_left == 0;
        if (ends || k + 1 == n_tiles) {
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) l += __shfl_xor_sync(~0u, l, d);
            if (x == 0) {
                s_m[h] = m;
                s_l[h] = l;
            }
            __syncthreads();
            const int32_t kvh = s_cur.seg / sets, first = s_cur.seg % sets * kLatentHeads, head0 = kvh * group + first;
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
                        *reinterpret_cast<uint4 *>(a.out + s_cur.r * a.out_stride + ((int64_t)(head0 + qh) * a.v_dim + d) * 2) = y;
                    }
                if (a.lse && threadIdx.x < heads)
                    a.lse[(int64_t)s_cur.r * a.n_q_heads + head0 + threadIdx.x] =
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
                if (begun && threadIdx.x == 0)
                    opened = OpenSegment{s_cur.r, s_cur.seg,
                                         batch.split.cta_of(s_cur.seg_begin(segs) + s_cur.tiles - 1) - (int32_t)blockIdx.x + 1, 0};
            }
        }
        if (k + 1 < n_tiles) {
            __syncthreads();                                       // nobody reads this stage, or s_cur, any more
            if (k + 2 < n_tiles) copy_rows(stage);
            if (k + 3 < n_tiles) lookup();
            if (ends) {
                if (threadIdx.x == 0) {
                    s_cur.tile = s_cur.tiles - 1;                  // only kept for the segment's ends
                    int64_t x = 0;
                    s_cur.next(a, segs, x);
                }
                __syncthreads();
                begun = true;
                tiles_left = s_cur.tiles;
                load_q();
            }
        }
    }
    if (s_timeout && threadIdx.x == 0) atomicAdd(a.pool.skipped + 1, 1ull);
    if (threadIdx.x == 0) open[blockIdx.x] = s_timeout ? OpenSegment{0, 0, 0, 0} : opened;
}

// Joins the segments that go over several CTAs. Up to kJoinFew pieces a thread joins a float4 of the sums by itself, 256 at a time;
// of more pieces 64 float4s at a time, four groups of 64 threads taking every fourth piece.
// Bound by three round trips to L2: the open segments, kept in shared memory with their places, then maxima, sums and results
// all at once. One request of 32768 8-bit latents, 152 pieces: 17.7 us, 4 more with the maxima first.
constexpr int kJoinThreads = 256, kJoinSlices = kLatentFloat4 / 64, kJoinCtas = 2;      // CTAs per SM: 8 start 1 us later, 1 takes 2 us longer
constexpr int kJoinList = 512;                                                          // at least the CTAs of the first kernel
constexpr int kJoinFew = 8;

template <int IO> __global__ void __launch_bounds__(kJoinThreads) kvx_attend_latent_join(const __grid_constant__ AttendArgs a, int ctas) {
    __shared__ OpenSegment s_list[kJoinList];
    __shared__ int32_t s_count[kJoinList / 32];
    __shared__ float4 s_o[4][64];
    __shared__ float s_top[4][64], s_sum[4][64];
    wait_for_earlier();
    const OpenSegment *const open = (const OpenSegment *)a.scratch;
    const uint8_t *const parts = a.scratch + kScratchCounters * sizeof(uint32_t);
    const int32_t group = a.n_q_heads / a.n_kv_heads, sets = (group + kLatentHeads - 1) / kLatentHeads;
    int n_open;
    {                                                              // in order: every CTA has to number them alike
        constexpr int kWarps = kJoinThreads / 32;
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
        OpenSegment seg[kJoinList / kJoinThreads];
        uint32_t found[kJoinList / kJoinThreads];
#pragma unroll
        for (int i = 0; i < kJoinList / kJoinThreads; ++i) {
            const int c = i * kJoinThreads + threadIdx.x;
            seg[i] = c < ctas ? open[c] : OpenSegment{0, 0, 0, 0};
            seg[i].cta = c;
            found[i] = __ballot_sync(~0u, seg[i].pieces > 0);
            if (lane == 0) s_count[i * kWarps + w] = __popc(found[i]);
        }
        __syncthreads();
        static_assert(kJoinList / 32 <= 32, "a count per lane");
        const int32_t mine = lane < kJoinList / 32 ? s_count[lane] : 0;
        int32_t upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t x = __shfl_up_sync(~0u, upto, d);
            if (lane >= d) upto += x;
        }
        n_open = __shfl_sync(~0u, upto, 31);
#pragma unroll
        for (int i = 0; i < kJoinList / kJoinThreads; ++i) {
            const int32_t before = __shfl_sync(~0u, upto - mine, i * kWarps + w);
            if (seg[i].pieces > 0) s_list[before + __popc(found[i] & ((1u << lane) - 1))] = seg[i];
        }
        __syncthreads();
    }
    // float4 f of the sums of one segment: query head, element, and the outputs
    auto head_of = [](int f) { return (f >> 7 & 1) * 8 + 2 * (f & 3) + (f >> 6 & 1); };
    auto element_of = [](int f) { return (f >> 8) * 64 + (f >> 2 & 7) * 8 + (f >> 5 & 1) * 4; };
    auto used = [&](const OpenSegment &seg, int f) {
        return seg.seg % sets * kLatentHeads + head_of(f) < group && element_of(f) < a.v_dim;
    };
    auto put = [&](const OpenSegment &seg, int f, float4 o, float top, float l) {
        const int q = head_of(f), d = element_of(f);
        const int32_t in_group = seg.seg % sets * kLatentHeads + q, head = seg.seg / sets * group + in_group;
        if (!used(seg, f)) return;
        const float inv = l == 0.0f ? 0.0f : a.v_scale / l;
        *reinterpret_cast<uint2 *>(a.out + seg.r * a.out_stride + ((int64_t)head * a.v_dim + d) * 2) =
            make_uint2(pack<IO>(o.x * inv, o.y * inv), pack<IO>(o.z * inv, o.w * inv));
        if (a.lse && d == 0) a.lse[(int64_t)seg.r * a.n_q_heads + head] = l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
    };
    for (int item = blockIdx.x; item < n_open * (kLatentFloat4 / kJoinThreads); item += gridDim.x) {
        const OpenSegment seg = s_list[item / (kLatentFloat4 / kJoinThreads)];
        const int f = item % (kLatentFloat4 / kJoinThreads) * kJoinThreads + threadIdx.x, q = head_of(f);
        if (seg.pieces > kJoinFew || !used(seg, f)) continue;
        const uint8_t *const first = parts + (size_t)(2 * seg.cta + 1) * kLatentPartial;         // the others: slot 0 of the CTAs after it
        float4 y[kJoinFew];
        float m[kJoinFew], s[kJoinFew], top = -INFINITY, l = 0.0f;
#pragma unroll
        for (int x = 0; x < kJoinFew; ++x) {
            const uint8_t *const p = x ? first + (size_t)(2 * x - 1) * kLatentPartial : first;
            m[x] = -INFINITY;
            if (x < seg.pieces) {
                y[x] = __ldcg((const float4 *)p + f);
                m[x] = __ldcg((const float *)(p + kLatentFloat4 * 16) + q);
                s[x] = __ldcg((const float *)(p + kLatentFloat4 * 16) + kLatentHeads + q);
            }
            top = fmaxf(top, m[x]);
        }
        const float ref = top == -INFINITY ? 0.0f : top;
        float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int x = 0; x < kJoinFew; ++x)
            if (x < seg.pieces) {
                const float z = fast_exp2(m[x] - ref);
                l += z * s[x];
                o.x += z * y[x].x;
                o.y += z * y[x].y;
                o.z += z * y[x].z;
                o.w += z * y[x].w;
            }
        put(seg, f, o, top, l);
    }
    const int f64 = threadIdx.x & 63, part = threadIdx.x >> 6;
    for (int item = blockIdx.x; item < n_open * kJoinSlices; item += gridDim.x) {
        const OpenSegment seg = s_list[item / kJoinSlices];
        const int f = item % kJoinSlices * 64 + f64, q = head_of(f);
        if (seg.pieces <= kJoinFew) continue;
        const uint8_t *const first = parts + (size_t)(2 * seg.cta + 1) * kLatentPartial;
        float top = -INFINITY, l = 0.0f;
        float4 o = make_float4(0, 0, 0, 0);
        for (int x0 = used(seg, f) ? part : seg.pieces; x0 < seg.pieces; x0 += 4 * kJoinFew) {
            float4 y[kJoinFew];
            float m[kJoinFew], s[kJoinFew], up = top;
#pragma unroll
            for (int k = 0; k < kJoinFew; ++k) {
                const int x = x0 + 4 * k;
                const uint8_t *const p = x ? first + (size_t)(2 * x - 1) * kLatentPartial : first;
                m[k] = -INFINITY;
                if (x < seg.pieces) {
                    y[k] = __ldcg((const float4 *)p + f);
                    m[k] = __ldcg((const float *)(p + kLatentFloat4 * 16) + q);
                    s[k] = __ldcg((const float *)(p + kLatentFloat4 * 16) + kLatentHeads + q);
                }
            }
#pragma unroll
            for (int k = 0; k < kJoinFew; ++k) up = fmaxf(up, m[k]);
            const float ref = up == -INFINITY ? 0.0f : up, old = fast_exp2(top - ref);
            top = up;
            l *= old;
            o = make_float4(o.x * old, o.y * old, o.z * old, o.w * old);
#pragma unroll
            for (int k = 0; k < kJoinFew; ++k)
                if (x0 + 4 * k < seg.pieces) {
                    const float z = fast_exp2(m[k] - ref);
                    l += z * s[k];
                    o.x += z * y[k].x;
                    o.y += z * y[k].y;
                    o.z += z * y[k].z;
                    o.w += z * y[k].w;
                }
        }
        s_o[part][f64] = o;
        s_top[part][f64] = top;
        s_sum[part][f64] = l;
        __syncthreads();
        if (part == 0) {
            float up = top;
#pragma unroll
            for (int i = 1; i < 4; ++i) up = fmaxf(up, s_top[i][f64]);
            const float ref = up == -INFINITY ? 0.0f : up;
            l = 0.0f;
            o = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 y = s_o[i][f64];
                const float z = fast_exp2(s_top[i][f64] - ref);
                l += z * s_sum[i][f64];
                o = make_float4(o.x + z * y.x, o.y + z * y.y, o.z + z * y.z, o.w + z * y.w);
            }
            put(seg, f, o, up, l);
        }
        __syncthreads();                                           // the parts are free again
    }
}

size_t latent_scratch_bytes(int32_t sms) { return kScratchCounters * sizeof(uint32_t) + (size_t)4 * sms * kLatentPartial; }

cudaError_t launch_latent_join(const AttendArgs &a, int32_t io, int ctas, int32_t sms, cudaStream_t stream) {
    if (ctas > kJoinList) return cudaErrorInvalidValue;
    return launch_after(io == KVX_BF16 ? kvx_attend_latent_join<KVX_BF16> : kvx_attend_latent_join<KVX_F16>, dim3(kJoinCtas * sms),
                        kJoinThreads, 0, stream, a, ctas);
}

template <class S> static cudaError_t launch(const AttendArgs &a, int32_t sms, cudaStream_t stream) {
    static std::atomic<uint64_t> asked;
    cudaError_t e = allow_shared(kvx_attend_latent<S>, S::BYTES, a.device, asked);
    if (e == cudaSuccess) e = launch_after(kvx_attend_latent<S>, dim3(2 * sms), kLatentThreads, S::BYTES, stream, a);
    return e != cudaSuccess ? e : launch_latent_join(a, S::IO, 2 * sms, sms, stream);
}

cudaError_t launch_attend_latent(const AttendArgs &a, int32_t vt, int32_t io, int32_t sms, cudaStream_t stream) {
    if (a.row_maps) return launch_latent_tensor(a, vt, io, sms, stream);
    if (vt == KVX_BF16) return launch<LatentShape<KVX_BF16, KVX_BF16>>(a, sms, stream);
    if (vt == KVX_F16) return launch<LatentShape<KVX_F16, KVX_F16>>(a, sms, stream);
    return io == KVX_BF16 ? launch<LatentShape<KVX_E4M3, KVX_BF16>>(a, sms, stream) : launch<LatentShape<KVX_E4M3, KVX_F16>>(a, sms, stream);
}

}  // namespace kvx
