// kvx_cache_attend over one plane of 8-bit latents, on the tcgen05 tensor pipe.
//
// The 8-bit codes are multiplied as they are, so nothing of the cache passes through registers: a tile of
// 128 positions is brought into shared memory by TMA in 128-byte swizzled chunks of 128 elements, and
// serves twice as operand A: by rows (K-major) for the scores
// S = K Q^T, 128 positions x 48, and by columns (MN-major) for the sums O^T += V^T P, four times 128
// elements x 48. What is not 8 bits wide is split into three codes with a spacing of 2^5, a column each:
//   x = c1 + c2 / 2^5 + c3 / 2^10,  each the nearest code of what is left,
// 12 significant bits and more, exact for bf16 queries down to 2^-18 of a query's largest element; so 16
// query heads make 48 columns. Their sums stand in TMEM apart and are put together in 32 bits.
//
// Queries are brought to a largest element in [2^7, 2^8) by a power of two. Weights are taken against a
// maximum that moves only when a score passes it by more than 2^kSlack, so that O in TMEM is hardly ever
// rescaled; times 2^5 they stay within the codes' range.
//
// Rows come in boxes of as many as a page holds in a row (the common divisor of the page and the tile);
// boxes that begin or end a sequence, and pages that 4 does not divide, are gathered four rows at a time,
// since a row that is not live has to read as zero. Gathers alone took 58 clocks each, 4.9 us a tile.
//
// Shared memory bounds the products, at 128 bytes a clock: a position is written once (576 bytes) and read
// twice (576 + 512), and the narrow operands add 400: 16 clocks an SM, where the memory takes 25. So what
// counts is that the copies never stop. Two tiles fit, and a tile's way (copy 1.9 us, scores 0.6, softmax
// 0.5, sums 0.4) is longer than the memory's time for two (3.3 us): each of the five chunks is therefore
// copied as soon as its sums are done, by a warp of its own, and multiplied as soon as it is there.
//
// Measured, 16 query heads: 64 sessions of 2048 to 32768 positions 122 us (644 MB; 1.7 us a tile, 0.97 of the
// copy rate, while it streams), 128 requests of 8000 115 us, 5.2 TB/s. Steps on the way: four rows a gather
// 408 us; boxes of a page's runs 167; chunk by chunk, products from a converged warp instead of one lane's
// branch (18 products 0.6 us, not 2.5) 153; eight softmax warps 146; a lighter join 140; a copying warp per
// chunk, and scores and sums from two warps 123. Prefetching the next tiles into L2 cost 8 to 17 us.
#include "kvx_latent.cuh"

namespace kvx {

constexpr int kTile = 128;                                     // positions
constexpr int kSoftThreads = 256;                              // warps 0-7: softmax and outputs, half of the query heads each four
constexpr int kCodeThreads = kSoftThreads + 7 * 32;            // 8, 9: products of the scores, of the sums; 10-14: copies, a chunk each
constexpr int kMine = kLatentHeads / 2;                        // query heads of a softmax thread
constexpr int kChunk = kTile * 128, kStage = 4 * kChunk + kTile * 64;   // 4 chunks of 128 elements, one of 64
constexpr int kChunks = 5;                                     // the last one is used up by the scores, the others in their order by the sums
constexpr int kTerms = 3, kCols = kTerms * kLatentHeads;
constexpr int kQueryBytes = kCols * kCacheMaxLatent, kWeightBytes = kCols * kTile;
constexpr int kOffQuery = 2 * kStage, kOffWeight = kOffQuery + kQueryBytes, kCodeBytes = kOffWeight + 2 * kWeightBytes;
constexpr float kSpacing = 32.0f;
constexpr float kSlack = 3.0f;                                 // in powers of two
constexpr float kWeightUp = 32.0f;                             // 2^(kSlack + 5) is within the codes' 448
constexpr uint32_t kColScores = 0, kColSums = 128, kTmemCols = 512;      // two buffers of scores 64 columns apart, then 4 x 48
constexpr int kCodeSwitch = 1;                                 // places of the line that a change of segment counts

// Shared memory operands: start, the two strides, swizzle (0 none, 2 of 128 bytes, 4 of 64 bytes).
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t leading, uint32_t stride, uint32_t swizzle) {
    return (uint64_t)(addr >> 4 & 0x3fff) | (uint64_t)(leading >> 4) << 16 | (uint64_t)(stride >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)swizzle << 61;
}
// 128 x 48 products of e4m3 codes with 32-bit sums; both operands by rows, or both by columns.
constexpr uint32_t kIdescRows = 1u << 4 | (kCols / 8) << 17 | (kTile / 16) << 24;
constexpr uint32_t kIdescCols = kIdescRows | 1u << 15 | 1u << 16;

// Issued by one lane of a converged warp, always the same: the operands are uniform then, and 18 products go out in 0.6 us
// instead of 2.5 from a branch of one lane.
__device__ __forceinline__ void tensor_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n.reg .pred p, e;\nsetp.ne.u32 p, %4, 0;\nelect.sync _|e, 0xffffffff;\n"
                 "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
                 : "memory");
}
__device__ __forceinline__ void tensor_commit(uint64_t *bar) {
    asm volatile("{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(shared_addr(bar)) : "memory");
}
__device__ __forceinline__ void tensor_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tensor_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 8 columns of this warp's 32 rows of TMEM.
__device__ __forceinline__ void tmem_load(uint32_t (&x)[kMine], uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]) : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_store(const uint32_t (&x)[kMine], uint32_t at) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
                 "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(shared_addr(bar)) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Barrier of the softmax warps, with the disjunction of a condition.
__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t y;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 q, %1, 0;\nbarrier.cta.red.or.pred p, 1, %2, q;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(y) : "r"((uint32_t)x), "n"(kSoftThreads) : "memory");
    return y;
}

// Codes of two values, and what is left of them, times the spacing.
__device__ __forceinline__ uint32_t take_codes(float &x, float &y) {
    uint16_t c;
    uint32_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(c) : "f"(x), "f"(y));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    const float2 f = unpack<KVX_F16>(h);
    x = (x - f.x) * kSpacing;
    y = (y - f.y) * kSpacing;
    return c;
}

// 8 values, one per query head, over the 32 lanes of the warp: the result is for head lane / 4.
template <class Op> __device__ __forceinline__ float reduce_heads(float (&v)[kMine], Op op) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = kMine / 2; n; n >>= 1) {
        const bool up = lane & 4 * n;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = op(keep, __shfl_xor_sync(~0u, give, 4 * n));
        }
    }
    v[0] = op(v[0], __shfl_xor_sync(~0u, v[0], 2));
    return op(v[0], __shfl_xor_sync(~0u, v[0], 1));
}

template <int IO> __global__ void __launch_bounds__(kCodeThreads, 1)
kvx_attend_latent_codes(const __grid_constant__ AttendArgs a, const __grid_constant__ RowMaps maps) {
    using Line = Place<kTile, kCodeSwitch>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_full[2][kChunks], s_free[2][kChunks];           // chunk by chunk
    __shared__ __align__(8) uint64_t s_scored[2], s_weighed[2], s_queried, s_drained[2];
    __shared__ uint8_t s_live[3][32];                              // live positions, four a byte
    __shared__ __align__(16) float s_red[4][kLatentHeads];
    __shared__ float s_scale[kLatentHeads];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int32_t s_failed;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t group = a.n_q_heads / a.n_kv_heads, sets = (group + kLatentHeads - 1) / kLatentHeads, segs = a.n_kv_heads * sets;

    if (threadIdx.x == 0) {                                        // what touches no memory, while the kernel before still runs
        s_failed = 0;
        for (int i = 0; i < 2; ++i) {
            for (int c = 0; c < kChunks; ++c) {
                asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_addr(&s_full[i][c])) : "memory");
                asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_addr(&s_free[i][c])) : "memory");
            }
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_addr(&s_scored[i])) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_addr(&s_drained[i])) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_addr(&s_weighed[i])), "n"(kSoftThreads) : "memory");
        }
        asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_addr(&s_queried)), "n"(kSoftThreads) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (w == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_addr(&s_tmem)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tensor_fence_before();
    }
    if (w == 10 && lane == 0)
        for (const CUtensorMap *m : {&maps.run128, &maps.run64}) asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    wait_for_earlier();
    OpenSegment *const open = (OpenSegment *)a.scratch;
    uint8_t *const parts = a.scratch + kScratchCounters * sizeof(uint32_t);
    const Batch<kTile, kCodeThreads / 32, 1, kCodeSwitch> batch(a, segs);
    const bool works = (int32_t)blockIdx.x < batch.split.ctas;
    const int64_t c_begin = works ? batch.split.begin(blockIdx.x) : 0, c_end = works ? batch.split.begin(blockIdx.x + 1) : 0;
    int64_t x0 = c_begin;
    Line begin = {};
    if (works) begin = batch.locate(a, segs, x0);
    __syncthreads();
    tensor_fence_after();
    const uint32_t tmem = s_tmem;
    // A wait of any role: false when it, or another role's, ran out. Copies and products then stop; the softmax warps, which
    // meet at barriers, go through their tiles without waiting any more.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (s_failed) return false;
        if (wait_full(bar, parity & 1)) return true;
        s_failed = 1;
        return false;
    };
    OpenSegment opened = {0, 0, 0, 0};

    if (x0 >= c_end) {
        // nothing, or nothing but the end of a segment
    } else if (w == 8) {                                           // products of the scores, chunk by chunk as they arrive
        const uint32_t smem0 = shared_addr(smem);                  // operands at their start; the rest are constants, in 16 bytes
        const uint64_t keys = operand(smem0, 16, 1024, 2), keys_last = operand(smem0 + 4 * kChunk, 16, 512, 4);
        const uint64_t queries = operand(smem0 + kOffQuery, (kCols / 8) * 128, 128, 0);
        Line at = begin;
        int64_t x = x0;
        int switches = 0;
        bool ok = true, first = true;
        for (int j = 0; ok && x < c_end; ++j) {
            const uint64_t stage = (j & 1) * (kStage / 16);
            const uint32_t d = tmem + kColScores + (j & 1) * 64;
            if (j >= 2) {                                          // the scores before are read
                ok = __all_sync(~0u, wait(&s_weighed[j & 1], (j - 2) >> 1));
                tensor_fence_after();
            }
            if (ok && first) ok = __all_sync(~0u, wait(&s_queried, switches++));
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int c = (i + 4) % kChunks;
                if (!ok || !(ok = __all_sync(~0u, wait(&s_full[j & 1][c], j >> 1)))) break;
#pragma unroll
                for (int y = 0; y < (c < 4 ? 4 : 2); ++y)
                    tensor_mma(d, (c < 4 ? keys + c * (kChunk / 16) : keys_last) + stage + y * 2, queries + (c * 8 + y * 2) * (kCols / 8) * 8, kIdescRows,
                               i > 0 || y > 0);
                if (c == 4) tensor_commit(&s_free[j & 1][4]);
            }
            if (ok) tensor_commit(&s_scored[j & 1]);
            at.next(a, segs, x);
            first = at.tile == 0;
        }
        if (!ok) {                                                 // no product outlives the CTA
            tensor_commit(&s_drained[0]);
            wait_full(&s_drained[0], 0);
        }
    } else if (w == 9) {                                           // products of the sums
        const uint32_t smem0 = shared_addr(smem);
        const uint64_t values = operand(smem0, 16, 1024, 2), weights = operand(smem0 + kOffWeight, 128, kTile * 16, 0);
        Line at = begin;
        int64_t x = x0;
        bool ok = true, first = true;
        for (int j = 0; x < c_end; ++j) {
            if (!(ok = __all_sync(~0u, wait(&s_weighed[j & 1], j >> 1)))) break;
            tensor_fence_after();
            const uint64_t v = values + (j & 1) * (kStage / 16), p = weights + (j & 1) * (kWeightBytes / 16);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tensor_mma(tmem + kColSums + c * kCols, v + c * (kChunk / 16) + i * 256, p + i * 32, kIdescCols, !first || i > 0);
                tensor_commit(&s_free[j & 1][c]);
            }
            at.next(a, segs, x);
            first = at.tile == 0;
        }
        if (!ok) {
            tensor_commit(&s_drained[1]);
            wait_full(&s_drained[1], 0);
        }
    } else if (w < 8) {                                            // softmax and outputs
        // a thread has a position (an element, of the outputs) and 8 query heads
        const int here = (w & 3) * 32 + lane, h0 = w >> 2 << 3;
        const uint32_t lanes = tmem + ((uint32_t)(w & 3) << 21) + h0;          // this warp's 32 rows, its first column
        float m[kMine], l[kMine], scale[kMine];
        // Queries of a segment as codes, and what its scores are to be multiplied by.
        auto query = [&](const Line &p) {
            const int h = threadIdx.x >> 4, part = threadIdx.x & 15;
            const int32_t kvh = p.seg / sets, in_group = p.seg % sets * kLatentHeads + h;
            const uint8_t *src = a.q + p.r * a.q_stride + ((int64_t)kvh * group + in_group) * a.head_dim * 2;
            const bool real = in_group < group;
            constexpr int kBlocks = (kCacheMaxLatent / 16 + 15) / 16;  // of 16 elements, for each of a head's 16 threads
            uint4 y[kBlocks][2];
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int d = (part + 16 * i) * 16 + k * 8;
                    y[i][k] = real && d < a.head_dim ? __ldg(reinterpret_cast<const uint4 *>(src + d * 2)) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    for (uint32_t z : {y[i][k].x, y[i][k].y, y[i][k].z, y[i][k].w}) {
                        const float2 f = unpack<IO>(z);
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            const int e = top > 0.0f && top < INFINITY ? max(-100, min(100, 7 - ilogbf(top))) : 0;
            const float up = __int_as_float((127 + e) << 23);
            if (part == 0) s_scale[h] = top < INFINITY ? a.scale * __int_as_float((127 - e) << 23) : NAN;     // an infinite query: NaN
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                const int b = part + 16 * i;
                if (b >= kCacheMaxLatent / 16) break;
                uint32_t codes[kTerms][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t z0 = k & 1 ? y[i][k >> 1].z : y[i][k >> 1].x, z1 = k & 1 ? y[i][k >> 1].w : y[i][k >> 1].y;
                    const float2 f0 = unpack<IO>(z0), f1 = unpack<IO>(z1);
                    float v[4] = {f0.x * up, f0.y * up, f1.x * up, f1.y * up};
#pragma unroll
                    for (int n = 0; n < kTerms; ++n) {
                        const uint32_t lo = take_codes(v[0], v[1]);
                        codes[n][k] = lo | take_codes(v[2], v[3]) << 16;
                    }
                }
#pragma unroll
                for (int n = 0; n < kTerms; ++n)                   // blocks of 8 columns x 16 elements
                    *(uint4 *)(smem + kOffQuery + (b * (kCols / 8) + n * 2 + (h >> 3)) * 128 + (h & 7) * 16) =
                        make_uint4(codes[n][0], codes[n][1], codes[n][2], codes[n][3]);
            }
            fence_async();
            arrive(&s_queried);
            softmax_any(false);
        };
        auto begin_segment = [&]() {
#pragma unroll
            for (int h = 0; h < kMine; ++h) {
                m[h] = -INFINITY;
                l[h] = 0.0f;
                scale[h] = s_scale[h0 + h];
            }
        };
        Line at = begin;
        int64_t x = x0;
        query(at);
        begin_segment();
        bool first = true, begun = at.seg_begin(segs) >= c_begin;  // the segment's first tile here; it begins in this CTA
        for (int j = 0;; ++j) {
            wait(&s_scored[j & 1], j >> 1);
            tensor_fence_after();
            float s[kMine];
            {
                uint32_t y[kTerms][kMine];
#pragma unroll
                for (int k = 0; k < kTerms; ++k) tmem_load(y[k], lanes + kColScores + (j & 1) * 64 + k * 16);
                tmem_load_wait();
                const bool live = s_live[j % 3][here >> 2] >> (here & 3) & 1;
#pragma unroll
                for (int h = 0; h < kMine; ++h) {
                    const float z = __uint_as_float(y[0][h]) + (__uint_as_float(y[1][h]) + __uint_as_float(y[2][h]) / kSpacing) / kSpacing;
                    s[h] = live ? z * scale[h] : -INFINITY;
                }
            }
            float over = -INFINITY;
#pragma unroll
            for (int h = 0; h < kMine; ++h) over = fmaxf(over, s[h] - m[h]);
            if (softmax_any(over > kSlack)) {                      // some maximum moves
                float v[kMine];
#pragma unroll
                for (int h = 0; h < kMine; ++h) v[h] = s[h];
                const float top = reduce_heads(v, [](float p, float q) { return fmaxf(p, q); });
                if (!(lane & 3)) s_red[w & 3][h0 + (lane >> 2)] = top;
                softmax_any(false);
                float old[kMine];
#pragma unroll
                for (int h = 0; h < kMine; ++h) {
                    const float up = fmaxf(m[h], fmaxf(fmaxf(s_red[0][h0 + h], s_red[1][h0 + h]), fmaxf(s_red[2][h0 + h], s_red[3][h0 + h])));
                    old[h] = fast_exp2(m[h] - (up == -INFINITY ? 0.0f : up));
                    m[h] = up;
                    l[h] *= old[h];
                }
                softmax_any(false);                                // s_red is free again
                if (!first) {
                    wait(&s_free[(j - 1) & 1][3], (j - 1) >> 1);
                    tensor_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 4 * kTerms; ++c) {
                        uint32_t y[kMine];
                        tmem_load(y, lanes + kColSums + c * 16);
                        tmem_load_wait();
#pragma unroll
                        for (int h = 0; h < kMine; ++h) y[h] = __float_as_uint(__uint_as_float(y[h]) * old[h]);
                        tmem_store(y, lanes + kColSums + c * 16);
                    }
                    tmem_store_wait();
                }
            }
            uint32_t codes[kTerms][2];
#pragma unroll
            for (int h = 0; h < kMine; h += 4) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = fast_exp2(s[h + i] - (m[h + i] == -INFINITY ? 0.0f : m[h + i]));
                    l[h + i] += v[i];
                    v[i] *= kWeightUp;
                }
#pragma unroll
                for (int k = 0; k < kTerms; ++k) {
                    const uint32_t lo = take_codes(v[0], v[1]);
                    codes[k][h / 4] = lo | take_codes(v[2], v[3]) << 16;
                }
            }
            if (j >= 2) wait(&s_free[j & 1][3], (j - 2) >> 1);
#pragma unroll
            for (int k = 0; k < kTerms; ++k)                       // blocks of 16 columns x 8 positions
                *(uint2 *)(smem + kOffWeight + (j & 1) * kWeightBytes + k * kTile * 16 + here * 16 + h0) = make_uint2(codes[k][0], codes[k][1]);
            fence_async();
            tensor_fence_before();
            arrive(&s_weighed[j & 1]);
            first = false;

            const bool ends = at.tile + 1 == at.tiles;
            Line nxt = at;
            nxt.next(a, segs, x);
            const bool more = x < c_end;
            if (!ends && more) {
                at = nxt;
                continue;
            }
            if (more) query(nxt);                                  // these scores are read, so the queries are free
            wait(&s_free[j & 1][3], j >> 1);
            tensor_fence_after();
            {
                float v[kMine];
#pragma unroll
                for (int h = 0; h < kMine; ++h) v[h] = l[h];
                const float sum = reduce_heads(v, [](float p, float q) { return p + q; });
                if (!(lane & 3)) s_red[w & 3][h0 + (lane >> 2)] = sum;
                softmax_any(false);
#pragma unroll
                for (int h = 0; h < kMine; ++h) l[h] = (s_red[0][h0 + h] + s_red[1][h0 + h]) + (s_red[2][h0 + h] + s_red[3][h0 + h]);
                softmax_any(false);
            }
            const bool whole = ends && begun;
            const int32_t in_group = at.seg % sets * kLatentHeads, head0 = at.seg / sets * group + in_group, heads = min(group - in_group, kLatentHeads);
            uint8_t *const part = parts + (size_t)(blockIdx.x * 2 + begun) * kLatentPartial;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t y[kTerms][kMine];
#pragma unroll
                for (int k = 0; k < kTerms; ++k) tmem_load(y[k], lanes + kColSums + c * kCols + k * 16);
                tmem_load_wait();
                const int d = c * 128 + here;
#pragma unroll
                for (int h = 0; h < kMine; ++h) {
                    const float z = (__uint_as_float(y[0][h]) + (__uint_as_float(y[1][h]) + __uint_as_float(y[2][h]) / kSpacing) / kSpacing) / kWeightUp;
                    if (!whole) __stcg((float *)part + partial_at(d, h0 + h), z);
                    else if (h0 + h < heads && d < a.v_dim)
                        ((uint16_t *)(a.out + at.r * a.out_stride))[(int64_t)(head0 + h0 + h) * a.v_dim + d] =
                            (uint16_t)pack<IO>(l[h] == 0.0f ? 0.0f : z * (a.v_scale / l[h]), 0.0f);
                }
            }
            tensor_fence_before();
#pragma unroll
            for (int h = 0; h < kMine; ++h)
                if (here == h) {
                    if (!whole) {
                        __stcg((float *)(part + kLatentFloat4 * 16) + h0 + h, m[h]);
                        __stcg((float *)(part + kLatentFloat4 * 16) + kLatentHeads + h0 + h, l[h]);
                    } else if (a.lse && h0 + h < heads)
                        a.lse[(int64_t)at.r * a.n_q_heads + head0 + h0 + h] = l[h] == 0.0f ? -INFINITY : (m[h] + log2f(l[h])) * kLn2;
                }
            if (!whole && begun)
                opened = OpenSegment{at.r, at.seg, batch.split.cta_of(at.seg_begin(segs) + at.tiles - 1) - (int32_t)blockIdx.x + 1, 0};
            if (!more) break;
            at = nxt;
            begin_segment();
            first = begun = true;
        }
    } else {                                                       // copies of a chunk
        const int c = w - 10;
        // A lane has a run of the tile, if there are as many, and four positions. Runs that are live or dead as a whole go in
        // boxes; the four positions of other runs by a gather.
        struct Rows {
            bool boxed, gathered;
            uint32_t row, y[4], live, col0;
        };
        const uint32_t run = (uint32_t)a.map_run, nothing = (uint32_t)a.map_rows;      // beyond the last row: reads as zeros
        auto look_up = [&](const Line &at) {
            Rows o;
            const int32_t kvh = at.seg / sets;
            const uint32_t first = (uint32_t)at.first, len = (uint32_t)at.len, tile0 = first / kTile * kTile + (uint32_t)at.tile * kTile;
            auto row_of = [&](uint32_t pos) {
                if (pos < first || pos >= len) return nothing;
                const uint32_t col = (__umulhi(pos, a.block_mul) + pos) >> a.block_shift, slot = pos - col * (uint32_t)a.pool.block_size;
                const int32_t blk = a.block_table[at.r * a.table_stride + col];
                if (blk < 0 || blk >= a.pool.n_blocks) {
                    if (at.seg == 0 && c == 0) atomicAdd(a.pool.skipped, 1ull);
                    return nothing;
                }
                return (uint32_t)blk * a.map_block + (uint32_t)kvh * a.map_head + slot;
            };
            auto whole = [&](uint32_t pos) { return run >= 4 && (pos + run <= first || pos >= len || (pos >= first && pos + run <= len)); };
            const uint32_t run0 = tile0 + lane * run, four0 = tile0 + 4 * lane, my_run = 4 * lane / run;
            o.col0 = (uint32_t)kvh * a.map_col;
            o.boxed = lane * run < kTile && whole(run0);
            o.gathered = !whole(tile0 + my_run * run);
            o.row = o.boxed ? row_of(run0) : nothing;
            o.live = __shfl_sync(~0u, o.row, my_run) != nothing ? 15 : 0;
            if (o.gathered) {
                o.live = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    o.y[k] = row_of(four0 + k);
                    o.live |= (uint32_t)(o.y[k] != nothing) << k;
                }
            }
            return o;
        };
        const CUtensorMap *const run_map = c < 4 ? &maps.run128 : &maps.run64, *const row_map = c < 4 ? &maps.row128 : &maps.row64;
        const uint32_t wide = c < 4 ? 128 : 64, bytes = wide * kTile;
        Line at = begin;
        int64_t x = x0;
        int issued = 0;
        Rows rows = look_up(at);
        for (; x < c_end; ++issued) {
            const int j = issued;
            if (!__all_sync(~0u, j < 2 || wait(&s_free[j & 1][c], (j - 2) >> 1))) break;
            const uint32_t bar = shared_addr(&s_full[j & 1][c]), to = shared_addr(smem + (j & 1) * kStage + c * kChunk);
            if (c == 0) {
                s_live[j % 3][lane] = (uint8_t)rows.live;          // tile j - 3 is through, its chunks were free
                __syncwarp();
            }
            if (lane == 0)                                         // a copy of another lane may count before: the phase waits for this
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
            if (rows.boxed)
                asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                                 to + lane * run * wide),
                             "l"(run_map), "r"(rows.col0 + c * 128), "r"(rows.row), "r"(bar)
                             : "memory");
            if (rows.gathered)
                asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
                             ::"r"(to + lane * 4 * wide), "l"(row_map), "r"(rows.col0 + c * 128), "r"(rows.y[0]), "r"(rows.y[1]), "r"(rows.y[2]),
                             "r"(rows.y[3]), "r"(bar)
                             : "memory");
            at.next(a, segs, x);
            if (x < c_end) rows = look_up(at);                     // while this one is under way
        }
        if (__any_sync(~0u, s_failed))                             // no copy outlives the CTA
            for (int j = max(0, issued - 2); j < issued; ++j) wait_full(&s_full[j & 1][c], j >> 1 & 1);
    }
    tensor_fence_before();
    __syncthreads();
    if (w == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    if (threadIdx.x == 0) {
        if (s_failed) atomicAdd(a.pool.skipped + 1, 1ull);
        open[blockIdx.x] = s_failed ? OpenSegment{0, 0, 0, 0} : opened;
    }
}

template <int IO> static cudaError_t launch(const AttendArgs &a, int32_t sms, cudaStream_t stream) {
    static std::atomic<uint64_t> asked;
    cudaError_t e = allow_shared(kvx_attend_latent_codes<IO>, kCodeBytes, a.device, asked);
    if (e == cudaSuccess) e = launch_after(kvx_attend_latent_codes<IO>, dim3(sms), kCodeThreads, kCodeBytes, stream, a, *a.row_maps);
    return e != cudaSuccess ? e : launch_latent_join(a, IO, sms, sms, stream);
}

cudaError_t launch_latent_codes(const AttendArgs &a, int32_t io, int32_t sms, cudaStream_t stream) {
    return io == KVX_BF16 ? launch<KVX_BF16>(a, sms, stream) : launch<KVX_F16>(a, sms, stream);
}

}  // namespace kvx
