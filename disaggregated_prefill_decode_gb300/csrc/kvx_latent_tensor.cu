// kvx_cache_attend over one plane of latents, on the tcgen05 tensor pipe.
//
// Nothing of the cache passes through registers: a tile of 128 positions (64 of 16 bits, the same bytes) is
// brought into shared memory by TMA, in chunks of 128 elements whose rows are swizzled over 128 bytes, and
// serves twice as operand A: by rows (K-major) for the scores S = K Q^T, 128 positions x the query columns,
// and by columns (MN-major) for the sums O^T += V^T P, four times 128 elements x the weight columns.
//
// 8-bit latents are multiplied as the codes they are. What is not 8 bits wide is split into codes with a
// spacing of 2^5, a column each:
//   x = c1 + c2 / 2^5 + c3 / 2^10 (+ c4 / 2^15),  each the nearest code of what is left.
// A query is three: 14 bits, exact for bf16 down to 2^-18 of its largest element, which is brought into
// [2^7, 2^8) by a power of two; of bf16 queries of 32 heads two, exact down to 2^-14 and 2^-22 of the largest
// off below. A weight is four, which leave 2^-18 of it, or 2^-30 of the row's largest. With three (2^-14, 2^-25)
// thousands of weights that small were lost beside a large one, and outputs differed from 32-bit products by 1.4e-4
// (9.5e-5 now, which is the order of the sums); the fourth costs 16 heads 1 % of the time. 32 heads have no room in
// TMEM for four columns of sums (4 x 128 are all of it): their second code has the first one's scale and goes into
// the first one's sums, as a product of its own, and the third is 2^10 from it. That leaves the same of large
// and of the smallest weights, 2^-9 of one below 2^-15, and costs 7 to 10 % (64 x 8000: 82 us, 76 with three codes; 16 heads at
// a time with four columns 107, less slack for the maximum, to 2^-27, 87). f16 queries go 16 heads at a time.
// 16-bit latents take a query as it is, and a weight as two values whose sum leaves 2^-17 of it (f16: 2^-23, or
// 2^-36 of the largest). The columns' sums stand in TMEM apart and are put together in 32 bits. Weights are taken
// against a maximum that moves only when a score passes it by more than 2^kSlack, so that O in TMEM is hardly
// ever rescaled; times 2^5 they stay within the codes' range.
//
// 16 query heads go at a time, or 32 where a KV head has more than 16: the columns of 32 take TMEM
// whole, and the cache is read half as often. 64 requests of 8000, 32 heads: bf16 122 us with 32, 206 with 16
// (117 since).
//
// Rows come in boxes of as many as a page holds in a row (the common divisor of the page and the tile);
// boxes that begin or end a sequence, and pages that 4 does not divide, are gathered four rows at a time,
// since a row that is not live has to read as zero. Gathers alone took 58 clocks each, 4.9 us a tile.
//
// Shared memory bounds the products, at 128 bytes a clock: 128 positions of 8 bits are written once (576
// bytes each) and read twice (576 + 512), and the narrow operands of 16 heads add 480: 17 clocks an SM, where
// the memory takes 25. So what counts is that the copies never stop. Two tiles fit, and a tile's way (copy
// 1.9 us, scores 0.6, softmax 0.5, sums 0.4) is longer than the memory's time for two (3.3 us): each of the
// five chunks is therefore copied as soon as its sums are done, by a warp of its own, and multiplied as soon
// as it is there.
//
// Measured, 16 query heads, 8 bits: 64 sessions of 2048 to 32768 positions 116 us (644 MB; 1.7 us a tile, 0.97
// of the copy rate, while it streams), 128 requests of 8000 113 us, 5.2 TB/s; bf16: 64 requests of 8000 108
// us, 128 201 us, 5.9 TB/s, which warp products (kvx_latent.cu) took 144 and 270 for. Steps on the way, 8
// bits: four rows a gather 408 us; boxes of a page's runs 167; chunk by chunk, products from a converged warp
// instead of one lane's branch (18 products 0.6 us, not 2.5) 153; eight softmax warps 146; a lighter join
// 140; a copying warp per chunk, and scores and sums from two warps 123; no query and no scale kept in
// registers, 119 (no spills with 16 heads; 8 bits with 32 heads have 24 bytes); outputs four elements at a time, with
// no division for each, 116 (4 requests of 100: 11.7, from 14.1); a join in one pass 115; a fourth code of the weights, for
// their precision, 116. Prefetching the next tiles into L2 cost 8 to 17 us.
#include "kvx_latent.cuh"
#include "kvx_tensor.cuh"

namespace kvx {

constexpr int kSoftThreads = 256;                              // warps 0-7: softmax and outputs, half of the query heads each four
constexpr int kTensorThreads = kSoftThreads + 7 * 32;          // 8, 9: products of the scores, of the sums; 10-14: copies, a chunk each
constexpr int kChunks = 5;                                     // the last one is used up by the scores, the others in their order by the sums
constexpr float kSlack = 3.0f;                                 // in powers of two
constexpr uint32_t kColScores = 0, kColSums = 128, kTmemCols = 512;      // of TMEM: two buffers of scores, then 4 x S::WCOLS sums

template <int VT_, int IO_, int HEADS_> struct TensorShape {
    static constexpr int VT = VT_, IO = IO_, HEADS = HEADS_;       // HEADS: query heads at a time
    static constexpr bool F8 = VT == KVX_E4M3;
    static constexpr int ESZ = F8 ? 1 : 2;
    static constexpr int TILE = 128 / ESZ;                        // positions
    static constexpr int SUBS = ESZ;                              // 128-byte pieces of a row in a chunk of 128 elements
    static constexpr int SUB = TILE * 128, CHUNK = SUBS * SUB;    // the last chunk has 64 elements
    static constexpr int STAGE = 4 * CHUNK + CHUNK / 2;
    static constexpr int LAST = F8 ? 64 : 128;                    // bytes of a row in the last chunk
    static constexpr bool WIDE = F8 && HEADS > 16;                // the second code of a weight shares the first one's sums
    static constexpr int QTERMS = !F8 ? 1 : WIDE ? 2 : 3, WTERMS = F8 ? 4 : 2;   // values of a query, of a weight
    static constexpr int SUMS = WIDE ? 3 : WTERMS;                // columns of a query head in the sums
    static constexpr int QCOLS = QTERMS * HEADS, WCOLS = SUMS * HEADS;
    // A weight's k-th value: what is left of it is multiplied by, and its place; a query's codes are 2^5 apart.
    static __host__ __device__ constexpr float spacing(int k) { return !WIDE ? 32.0f : k == 0 ? 1.0f : k == 1 ? 1024.0f : 32.0f; }
    static __host__ __device__ constexpr int place(int k) { return !WIDE || k == 0 ? k : k == 1 ? 3 : k - 1; }
    static __host__ __device__ constexpr float sum_spacing(int k) { return !F8 ? 1.0f : WIDE && k == 0 ? 1024.0f : 32.0f; }   // of sums k and k + 1
    static constexpr int QUERY = QCOLS * kCacheMaxLatent * ESZ, WEIGHT = WTERMS * HEADS * TILE * ESZ;
    static constexpr int OFF_QUERY = 2 * STAGE, OFF_WEIGHT = OFF_QUERY + QUERY, BYTES = OFF_WEIGHT + 2 * WEIGHT;
    // Of the weights, up to 2^kSlack: 2^(3 + 5) is within the codes' 448, 2^(3 + 12) within f16, whose two values then have a
    // step of 2^-36 (times 1, weights below 2^-25 were lost).
    static constexpr float UP = F8 ? 32.0f : VT == KVX_F16 ? 4096.0f : 1.0f;
    // Places of the line that a change of segment counts: queries, then outputs. 300 requests of up to 1000 8-bit latents: 16 heads
    // 42.3 us with 1, 39.9 with 2, 39.5 with 3; 32 heads 65.2, 59.8, 57.0; long segments the same.
    static constexpr int SWITCH = HEADS / 16 + 1;
    static constexpr int ROWS = F8 ? 32 : 16;                     // of the scores in a warp's lanes of TMEM: 64 rows leave half free
    static constexpr int HALF = HEADS / 2;                        // query heads of four softmax warps
    static constexpr int MINE = HALF * ROWS / 32;                 // of a thread's scores
    static_assert(!WIDE || IO == KVX_BF16, "two codes hold a bf16 query, not an f16 one");
    static_assert(QCOLS <= 64 && kColSums + 4 * WCOLS <= kTmemCols && MINE * ESZ % 8 == 0, "room in TMEM, weights in pieces of 8 or 16 bytes");
    // M x N products with 32-bit sums: both operands by rows, or both by columns; bf16 is type 1, e4m3 and f16 are 0
    static constexpr uint32_t IDESC = 1u << 4 | (VT == KVX_BF16 ? 1u << 7 | 1u << 10 : 0);
    static constexpr uint32_t IDESC_ROWS = IDESC | (QCOLS / 8) << 17 | (TILE / 16) << 24;
    static constexpr uint32_t IDESC_COLS = IDESC | (WCOLS / 8) << 17 | (128 / 16) << 24 | 1u << 15 | 1u << 16;
    static constexpr uint32_t IDESC_SECOND = IDESC | (HEADS / 8) << 17 | (128 / 16) << 24 | 1u << 15 | 1u << 16;
};

// Barrier of the softmax warps, with the disjunction of a condition.
__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t y;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 q, %1, 0;\nbarrier.cta.red.or.pred p, 1, %2, q;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(y) : "r"((uint32_t)x), "n"(kSoftThreads) : "memory");
    return y;
}

// Codes of two values, and what is left of them, times the spacing.
__device__ __forceinline__ uint32_t take_codes(float &x, float &y, float spacing) {
    uint16_t c;
    uint32_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(c) : "f"(x), "f"(y));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    const float2 f = unpack<KVX_F16>(h);
    x = (x - f.x) * spacing;
    y = (y - f.y) * spacing;
    return c;
}

// The same of two f16 values.
__device__ __forceinline__ uint32_t take_codes(__half2 &x) {
    uint16_t c;
    uint32_t h;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    x = __hmul2(__hsub2(x, *reinterpret_cast<const __half2 *>(&h)), __float2half2_rn(32.0f));
    return c;
}

// N values, one per query head, over a group of LANES lanes: the result is for head (lane of the group) / (LANES / N).
template <int LANES, int N, class Op> __device__ __forceinline__ float reduce_heads(float (&v)[N], Op op) {
    const int lane = threadIdx.x & 31;
    int d = LANES / 2;
#pragma unroll
    for (int n = N / 2; n; n >>= 1, d >>= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = op(keep, __shfl_xor_sync(~0u, give, d));
        }
    }
#pragma unroll
    for (int x = LANES / N / 2; x; x >>= 1) v[0] = op(v[0], __shfl_xor_sync(~0u, v[0], x));
    return v[0];
}

template <class S> __global__ void __launch_bounds__(kTensorThreads, 1)
kvx_attend_latent_tensor(const __grid_constant__ AttendArgs a, const __grid_constant__ RowMaps maps) {
    constexpr int VT = S::VT, IO = S::IO, QTERMS = S::QTERMS, WTERMS = S::WTERMS, HEADS = S::HEADS, HALF = S::HALF, MINE = S::MINE;
    constexpr bool F8 = S::F8;
    using Line = Place<S::TILE, S::SWITCH>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_full[2][kChunks], s_free[2][kChunks];           // chunk by chunk
    __shared__ __align__(8) uint64_t s_scored[2], s_weighed[2], s_queried, s_drained[2], s_never;
    __shared__ uint8_t s_live[3][32];                              // live positions, four a byte
    __shared__ __align__(16) float s_red[4][S::HEADS], s_scale[2][S::HEADS], s_old[S::HEADS], s_m[S::HEADS], s_l[S::HEADS], s_inverse[S::HEADS];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int32_t s_failed;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t group = a.n_q_heads / a.n_kv_heads, sets = (group + HEADS - 1) / HEADS, segs = a.n_kv_heads * sets;

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
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_addr(&s_never)) : "memory");
        asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_addr(&s_queried)), "n"(kSoftThreads) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (w == 10 && lane == 0)
        for (const CUtensorMap *m : {&maps.run128, &maps.run64}) asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    wait_for_earlier();
    if (w == 8) {                                                  // not before: a kernel that still runs may yet ask for this TMEM
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_addr(&s_tmem)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tensor_fence_before();
    }
    OpenSegment *const open = (OpenSegment *)a.scratch;
    uint8_t *const parts = a.scratch + kScratchCounters * sizeof(uint32_t);
    const Batch<S::TILE, kTensorThreads / 32, 1, S::SWITCH, 0> batch(a, segs);
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
        if (wait_full(bar, parity & 1, a.wait_ns)) return true;
        s_failed = 1;
        return false;
    };
    // Whether a part goes on: it does, but where the testing hook has it wait for what never comes.
    auto goes_on = [&](int part) { return a.stall != part || blockIdx.x != 0 || wait(&s_never, 0); };
    int issued = 0;                                                // copying warps: tiles
    OpenSegment opened = {0, 0, 0, 0};

    if (x0 >= c_end) {
        // nothing, or nothing but the end of a segment
    } else if (w == 8) {                                           // products of the scores, chunk by chunk as they arrive
        const uint32_t smem0 = shared_addr(smem);                  // operands at their start; the rest are constants, in 16 bytes
        const uint64_t keys = operand(smem0, 16, 1024, 2), keys_last = operand(smem0 + 4 * S::CHUNK, 16, 8 * S::LAST, F8 ? 4 : 2);
        const uint64_t queries = operand(smem0 + S::OFF_QUERY, (S::QCOLS / 8) * 128, 128, 0);
        Line at = begin;
        int64_t x = x0;
        int switches = 0;
        bool ok = __all_sync(~0u, goes_on(kStallScores)), first = true;
        for (int j = 0; ok && x < c_end; ++j) {
            const uint64_t stage = (j & 1) * (S::STAGE / 16);
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
                for (int y = 0; y < (c < 4 ? 4 * S::SUBS : 2 * S::SUBS); ++y)          // 32 bytes of the rows
                    tensor_mma<F8>(d, (c < 4 ? keys + c * (S::CHUNK / 16) : keys_last) + stage + y / 4 * (S::SUB / 16) + y % 4 * 2,
                                   queries + (c * 8 * S::SUBS + y * 2) * (S::QCOLS / 8) * 8, S::IDESC_ROWS, i > 0 || y > 0);
                if (c == 4) tensor_commit(&s_free[j & 1][4]);
            }
            if (ok) tensor_commit(&s_scored[j & 1]);
            at.next(a, segs, x);
            first = at.tile == 0;
        }
    } else if (w == 9) {                                           // products of the sums
        const uint32_t smem0 = shared_addr(smem);
        const uint64_t values = operand(smem0, F8 ? 16 : S::SUB, 1024, 2), weights = operand(smem0 + S::OFF_WEIGHT, 128, S::TILE * 16, 0);
        Line at = begin;
        int64_t x = x0;
        bool first = true;
        if (!__all_sync(~0u, goes_on(kStallSums))) x = c_end;
        for (int j = 0; x < c_end; ++j) {
            if (!__all_sync(~0u, wait(&s_weighed[j & 1], j >> 1))) break;
            tensor_fence_after();
            const uint64_t v = values + (j & 1) * (S::STAGE / 16), p = weights + (j & 1) * (S::WEIGHT / 16);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
#pragma unroll
                for (int i = 0; i < 4; ++i)                        // a quarter of the positions
                    tensor_mma<F8>(tmem + kColSums + c * S::WCOLS, v + c * (S::CHUNK / 16) + i * (S::SUB / 64), p + i * (S::TILE / 4), S::IDESC_COLS,
                                   !first || i > 0);
                if constexpr (S::WIDE)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tensor_mma<F8>(tmem + kColSums + c * S::WCOLS, v + c * (S::CHUNK / 16) + i * (S::SUB / 64),
                                       p + (S::WCOLS / 16) * S::TILE + i * (S::TILE / 4), S::IDESC_SECOND, true);
                tensor_commit(&s_free[j & 1][c]);
            }
            at.next(a, segs, x);
            first = at.tile == 0;
        }
    } else if (w < 8) {                                            // softmax and outputs
        // A thread has a position and MINE query heads of the scores, an element and HALF of the outputs. The scores of a
        // tile of 64 positions stand in half of the lanes, which hand half of the heads to the others.
        const int here = (w & 3) * 32 + lane, half0 = (w >> 2) * HALF;
        const int pos = (w & 3) * S::ROWS + lane % S::ROWS, h0 = half0 + lane / S::ROWS * MINE;
        const uint32_t lanes = tmem + ((uint32_t)(w & 3) << 21) + half0;       // this warp's 32 rows, its first column
        constexpr int kParts = kSoftThreads / HEADS;               // threads of a query
        float m[MINE], l[MINE];
        int turn = 0;                                              // of s_scale
        // Queries of a segment as codes, and what its scores are to be multiplied by.
        auto query = [&](const Line &p, int turn) {
            const int h = threadIdx.x / kParts, part = threadIdx.x % kParts;
            const int32_t kvh = p.seg / sets, in_group = p.seg % sets * HEADS + h;
            const uint8_t *src = a.q + p.r * a.q_stride + ((int64_t)kvh * group + in_group) * a.head_dim * 2;
            const bool real = in_group < group;
            if constexpr (F8) {
                constexpr int kBlocks = (kCacheMaxLatent / 16 + kParts - 1) / kParts;          // of 16 elements, for each of a head's threads
                auto read = [&](int i, uint4 (&y)[2]) {            // twice: kept in registers, they cost the softmax spills
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int d = (part + kParts * i) * 16 + k * 8;
                        y[k] = real && d < a.head_dim ? __ldg(reinterpret_cast<const uint4 *>(src + d * 2)) : make_uint4(0, 0, 0, 0);
                    }
                };
                uint4 y[2];
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) {
                    read(i, y);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        for (uint32_t z : {y[k].x, y[k].y, y[k].z, y[k].w}) {
                            const float2 f = unpack<IO>(z);
                            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                }
#pragma unroll
                for (int d = 1; d < kParts; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                const int e = top > 0.0f && top < INFINITY ? max(-126, min(100, 7 - ilogbf(top))) : 0;
                const float up = __int_as_float((127 + e) << 23);
                if (part == 0) s_scale[turn][h] = top < INFINITY ? a.scale * __int_as_float((127 - e) << 23) : NAN;     // an infinite query: NaN
                read(0, y);
#pragma unroll 1
                for (int i = 0; i < kBlocks; ++i) {
                    const int b = part + kParts * i;
                    if (b >= kCacheMaxLatent / 16) break;
                    uint4 after[2];
                    read(i + 1, after);
                    uint32_t codes[QTERMS][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t z0 = k & 1 ? y[k >> 1].z : y[k >> 1].x, z1 = k & 1 ? y[k >> 1].w : y[k >> 1].y;
                        const float2 f0 = unpack<IO>(z0), f1 = unpack<IO>(z1);
                        float v[4] = {f0.x * up, f0.y * up, f1.x * up, f1.y * up};
#pragma unroll
                        for (int n = 0; n < QTERMS; ++n) {
                            const uint32_t lo = take_codes(v[0], v[1], 32.0f);
                            codes[n][k] = lo | take_codes(v[2], v[3], 32.0f) << 16;
                        }
                    }
#pragma unroll
                    for (int n = 0; n < QTERMS; ++n)                   // blocks of 8 columns x 16 elements
                        *(uint4 *)(smem + S::OFF_QUERY + (b * (S::QCOLS / 8) + n * (HEADS / 8) + (h >> 3)) * 128 + (h & 7) * 16) =
                            make_uint4(codes[n][0], codes[n][1], codes[n][2], codes[n][3]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) y[k] = after[k];
                }
            } else {                                               // as they are, in blocks of 8 columns x 8 elements
#pragma unroll
                for (int b = part; b < kCacheMaxLatent / 8; b += kParts)
                    *(uint4 *)(smem + S::OFF_QUERY + (b * (S::QCOLS / 8) + (h >> 3)) * 128 + (h & 7) * 16) =
                        real && b * 8 < a.head_dim ? __ldg(reinterpret_cast<const uint4 *>(src + b * 16)) : make_uint4(0, 0, 0, 0);
            }
            fence_async();
            arrive(&s_queried);
            softmax_any(false);
        };
        auto begin_segment = [&]() {
#pragma unroll
            for (int h = 0; h < MINE; ++h) {
                m[h] = -INFINITY;
                l[h] = 0.0f;
            }
        };
        Line at = begin;
        int64_t x = x0;
        goes_on(kStallSoftmax);
        query(at, 0);
        begin_segment();
        bool first = true, begun = at.seg_begin(segs) >= c_begin;  // the segment's first tile here; it begins in this CTA
        for (int j = 0;; ++j) {
            wait(&s_scored[j & 1], j >> 1);
            tensor_fence_after();
            float s[MINE];
            {
                const bool live = s_live[j % 3][pos >> 2] >> (pos & 3) & 1;
                float z[HALF];
#pragma unroll
                for (int i = 0; i < HALF; i += 8) {
                    uint32_t y[QTERMS][8];
#pragma unroll
                    for (int k = 0; k < QTERMS; ++k) tmem_load(y[k], lanes + kColScores + (j & 1) * 64 + k * HEADS + i);
                    tmem_load_wait();
#pragma unroll
                    for (int h = 0; h < 8; ++h) {
                        z[i + h] = __uint_as_float(y[0][h]);
                        float rest = 0.0f;
#pragma unroll
                        for (int k = QTERMS - 1; k > 0; --k) rest = (__uint_as_float(y[k][h]) + rest) / 32.0f;
                        z[i + h] += rest;
                    }
                }
#pragma unroll
                for (int h = 0; h < MINE; ++h) {
                    if constexpr (F8) s[h] = z[h] * s_scale[turn][h0 + h];
                    else {
                        const float other = __shfl_sync(~0u, z[MINE + h], lane % S::ROWS);
                        s[h] = (lane < S::ROWS ? z[h] : other) * a.scale;
                    }
                    if (!live) s[h] = -INFINITY;
                }
            }
            float over = -INFINITY;
#pragma unroll
            for (int h = 0; h < MINE; ++h) over = fmaxf(over, s[h] - m[h]);
            constexpr int kLanes = S::ROWS / MINE;                 // that reduce_heads leaves a head's result in
            if (softmax_any(over > kSlack)) {                      // some maximum moves
                float v[MINE];
#pragma unroll
                for (int h = 0; h < MINE; ++h) v[h] = s[h];
                const float top = reduce_heads<S::ROWS>(v, [](float p, float q) { return fmaxf(p, q); });
                if (lane % kLanes == 0) s_red[w & 3][h0 + lane % S::ROWS / kLanes] = top;
                softmax_any(false);
                float old[MINE];
#pragma unroll
                for (int h = 0; h < MINE; ++h) {
                    const float up = fmaxf(m[h], fmaxf(fmaxf(s_red[0][h0 + h], s_red[1][h0 + h]), fmaxf(s_red[2][h0 + h], s_red[3][h0 + h])));
                    old[h] = fast_exp2(m[h] - (up == -INFINITY ? 0.0f : up));
                    m[h] = up;
                    l[h] *= old[h];
                    if (MINE < HALF && (w & 3) == 0 && lane % S::ROWS == 0) s_old[h0 + h] = old[h];
                }
                softmax_any(false);                                // s_red is free again
                if (!first) {
                    wait(&s_free[(j - 1) & 1][3], (j - 1) >> 1);
                    tensor_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 4 * S::SUMS; ++c)
#pragma unroll
                        for (int i = 0; i < HALF; i += 8) {
                            uint32_t y[8];
                            tmem_load(y, lanes + kColSums + c * HEADS + i);
                            tmem_load_wait();
#pragma unroll
                            for (int h = 0; h < 8; ++h) y[h] = __float_as_uint(__uint_as_float(y[h]) * (MINE < HALF ? s_old[half0 + i + h] : old[(i + h) % MINE]));
                            tmem_store(y, lanes + kColSums + c * HEADS + i);
                        }
                    tmem_store_wait();
                }
            }
            uint32_t terms[WTERMS][MINE * S::ESZ / 4];             // the heads' weights, term by term
#pragma unroll
            for (int h = 0; h < MINE; h += 4) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = fast_exp2(s[h + i] - (m[h + i] == -INFINITY ? 0.0f : m[h + i]));
                    l[h + i] += v[i];
                    v[i] *= S::UP;
                }
                if constexpr (F8) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t lo = take_codes(v[0], v[1], S::spacing(k));
                        terms[S::place(k)][h / 4] = lo | take_codes(v[2], v[3], S::spacing(k)) << 16;
                    }
                    __half2 y0 = __floats2half2_rn(v[0], v[1]), y1 = __floats2half2_rn(v[2], v[3]);   // 11 bits: a quarter of what the last code leaves
#pragma unroll
                    for (int k = 2; k < WTERMS; ++k) {
                        const uint32_t lo = take_codes(y0);
                        terms[S::place(k)][h / 4] = lo | take_codes(y1) << 16;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const uint32_t top = pack<VT>(v[i], v[i + 1]);
                        const float2 f = unpack<VT>(top);
                        terms[0][(h + i) / 2] = top;
                        terms[1][(h + i) / 2] = pack<VT>(v[i] - f.x, v[i + 1] - f.y);
                    }
                }
            }
            if (j >= 2) wait(&s_free[j & 1][3], (j - 2) >> 1);
#pragma unroll
            for (int k = 0; k < WTERMS; ++k) {                     // blocks of 16 bytes of columns x 8 positions
                const int col = (k * HEADS + h0) * S::ESZ;
                uint8_t *const to = smem + S::OFF_WEIGHT + (j & 1) * S::WEIGHT + col / 16 * S::TILE * 16 + pos * 16 + col % 16;
                if constexpr (MINE * S::ESZ == 8) *(uint2 *)to = make_uint2(terms[k][0], terms[k][1]);
                else *(uint4 *)to = make_uint4(terms[k][0], terms[k][1], terms[k][2], terms[k][3]);
            }
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
            if (more) query(nxt, turn ^ 1);                                  // these scores are read, so the queries are free
            wait(&s_free[j & 1][3], j >> 1);
            tensor_fence_after();
            {
                float v[MINE];
#pragma unroll
                for (int h = 0; h < MINE; ++h) {
                    v[h] = l[h];
                    if ((w & 3) == 0 && lane % S::ROWS == 0) s_m[h0 + h] = m[h];
                }
                const float sum = reduce_heads<S::ROWS>(v, [](float p, float q) { return p + q; });
                if (lane % kLanes == 0) s_red[w & 3][h0 + lane % S::ROWS / kLanes] = sum;
                softmax_any(false);
                if (threadIdx.x < HEADS) {
                    const float all = (s_red[0][threadIdx.x] + s_red[1][threadIdx.x]) + (s_red[2][threadIdx.x] + s_red[3][threadIdx.x]);
                    s_l[threadIdx.x] = all;
                    s_inverse[threadIdx.x] = all == 0.0f ? 0.0f : a.v_scale / all;
                }
                softmax_any(false);
            }
            const bool whole = ends && begun;
            const int32_t in_group = at.seg % sets * HEADS, head0 = at.seg / sets * group + in_group, heads = min(group - in_group, HEADS);
            uint16_t *const out = (uint16_t *)(a.out + at.r * a.out_stride) + (int64_t)head0 * a.v_dim;
            // partial results are of kLatentHeads heads: the second half of 32 goes where another CTA's would be
            auto part_of = [&](int h) { return parts + ((size_t)(blockIdx.x + h / kLatentHeads * gridDim.x) * 2 + begun) * kLatentPartial; };
#pragma unroll 1
            for (int c = 0; c < 4; ++c)
#pragma unroll 1
                for (int i = 0; i < HALF; i += 8) {
                    uint32_t y[S::SUMS][8];
#pragma unroll
                    for (int k = 0; k < S::SUMS; ++k) tmem_load(y[k], lanes + kColSums + c * S::WCOLS + k * HEADS + i);
                    tmem_load_wait();
                    float z[8];
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        z[n] = __uint_as_float(y[S::SUMS - 1][n]);
#pragma unroll
                        for (int k = S::SUMS - 2; k >= 0; --k) z[n] = __uint_as_float(y[k][n]) + z[n] / S::sum_spacing(k);
                        z[n] /= S::UP;
                    }
                    // among four lanes, from 8 heads of an element each to two heads of four elements
                    const int b0 = lane & 1, b1 = lane >> 1 & 1, d = c * 128 + (here & ~3);
                    float u[4][2], t[2][4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float keep = b0 ? z[4 + n] : z[n], got = __shfl_xor_sync(~0u, b0 ? z[n] : z[4 + n], 1);
                        u[n][0] = b0 ? got : keep;
                        u[n][1] = b0 ? keep : got;
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float keep = b1 ? u[2 + n][e] : u[n][e], got = __shfl_xor_sync(~0u, b1 ? u[n][e] : u[2 + n][e], 2);
                            t[n][e] = b1 ? got : keep;
                            t[n][2 + e] = b1 ? keep : got;
                        }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int h = half0 + i + b0 * 4 + b1 * 2 + n;
                        if (!whole) __stcg((float4 *)((float *)part_of(h) + partial_at(d, h % kLatentHeads)), make_float4(t[n][0], t[n][1], t[n][2], t[n][3]));
                        else if (h < heads && d < a.v_dim) {
                            const float inverse = s_inverse[h];
                            const bool none = s_l[h] == 0.0f;
                            *reinterpret_cast<uint2 *>(out + h * a.v_dim + d) =
                                none ? make_uint2(0, 0)
                                     : make_uint2(pack<IO>(t[n][0] * inverse, t[n][1] * inverse), pack<IO>(t[n][2] * inverse, t[n][3] * inverse));
                        }
                    }
                }
            tensor_fence_before();
            if (threadIdx.x < HEADS) {
                const int h = threadIdx.x;
                if (!whole) {
                    float *const ml = (float *)(part_of(h) + kLatentFloat4 * 16) + h % kLatentHeads;
                    __stcg(ml, s_m[h]);
                    __stcg(ml + kLatentHeads, s_l[h]);
                } else if (a.lse && h < heads)
                    a.lse[(int64_t)at.r * a.n_q_heads + head0 + h] = s_l[h] == 0.0f ? -INFINITY : (s_m[h] + log2f(s_l[h])) * kLn2;
            }
            if (!whole && begun)
                opened = OpenSegment{at.r, at.seg, batch.split.cta_of(at.seg_begin(segs) + at.tiles - 1) - (int32_t)blockIdx.x + 1, 0};
            if (!more) break;
            at = nxt;
            turn ^= 1;
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
            const uint32_t first = (uint32_t)at.first, len = (uint32_t)at.len, tile0 = first / S::TILE * S::TILE + (uint32_t)at.tile * S::TILE;
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
            o.boxed = lane * run < S::TILE && whole(run0);
            o.gathered = lane * 4 < S::TILE && !whole(tile0 + my_run * run);
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
        const bool narrow = F8 && c == 4;
        const CUtensorMap *const run_map = narrow ? &maps.run64 : &maps.run128, *const row_map = narrow ? &maps.row64 : &maps.row128;
        const uint32_t wide = narrow ? 64 : 128, subs = c < 4 ? S::SUBS : 1, bytes = wide * subs * S::TILE;
        Line at = begin;
        int64_t x = x0;
        if (c == 0 && !__all_sync(~0u, goes_on(kStallCopies))) x = c_end;
        Rows rows = look_up(at);
        for (; x < c_end; ++issued) {
            const int j = issued;
            if (!__all_sync(~0u, j < 2 || wait(&s_free[j & 1][c], (j - 2) >> 1))) break;
            const uint32_t bar = shared_addr(&s_full[j & 1][c]), chunk = shared_addr(smem + (j & 1) * S::STAGE + c * S::CHUNK);
            if (c == 0) {
                s_live[j % 3][lane] = (uint8_t)rows.live;          // tile j - 3 is through, its chunks were free
                __syncwarp();
            }
            if (lane == 0)                                         // a copy of another lane may count before: the phase waits for this
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
#pragma unroll
            for (int i = 0; i < S::SUBS; ++i) {
                if (i >= subs) break;
                const uint32_t to = chunk + i * S::SUB, col = rows.col0 + (c * S::SUBS + i) * 128;
                if (rows.boxed)
                    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                                     to + lane * run * wide),
                                 "l"(run_map), "r"(col), "r"(rows.row), "r"(bar)
                                 : "memory");
                if (rows.gathered)
                    asm volatile(
                        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
                        ::"r"(to + lane * 4 * wide), "l"(row_map), "r"(col), "r"(rows.y[0]), "r"(rows.y[1]), "r"(rows.y[2]), "r"(rows.y[3]), "r"(bar)
                        : "memory");
            }
            at.next(a, segs, x);
            if (x < c_end) rows = look_up(at);                     // while this one is under way
        }
    }
    tensor_fence_before();
    __syncthreads();
    if (s_failed) {                                                // no copy or product outlives the CTA, whoever's wait ran out
        if (w == 8 || w == 9) {
            tensor_commit(&s_drained[w - 8]);
            wait_full(&s_drained[w - 8], 0, kCacheWaitNs);
        } else if (w > 9)
            for (int j = max(0, issued - 2); j < issued; ++j) wait_full(&s_full[j & 1][w - 10], j >> 1 & 1, kCacheWaitNs);
        tensor_fence_before();
        __syncthreads();
    }
    if (w == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    if (threadIdx.x == 0) {
        if (s_failed) atomicAdd(a.pool.skipped + 1, 1ull);
        for (int i = 0; i < HEADS / kLatentHeads; ++i) {           // as segments of kLatentHeads
            const int32_t in_group = opened.seg % sets * HEADS + i * kLatentHeads, of_16 = (group + kLatentHeads - 1) / kLatentHeads;
            open[blockIdx.x + i * gridDim.x] =
                s_failed || in_group >= group ? OpenSegment{0, 0, 0, 0}
                                              : OpenSegment{opened.r, opened.seg / sets * of_16 + in_group / kLatentHeads, opened.pieces, 0};
        }
    }
}

template <class S> static cudaError_t launch(const AttendArgs &a, int32_t sms, cudaStream_t stream) {
    static std::atomic<uint64_t> asked;
    cudaError_t e = allow_shared(kvx_attend_latent_tensor<S>, S::BYTES, a.device, asked);
    if (e == cudaSuccess) e = launch_after(kvx_attend_latent_tensor<S>, dim3(sms), kTensorThreads, S::BYTES, stream, a, *a.row_maps);
    return e != cudaSuccess ? e : launch_latent_join(a, S::IO, S::HEADS / kLatentHeads * sms, sms, stream);
}

template <int VT, int IO> static cudaError_t launch_heads(const AttendArgs &a, int32_t sms, cudaStream_t stream) {
    if constexpr (VT != KVX_E4M3 || IO == KVX_BF16)                // f16 queries of 32 heads in three codes leave no room for the weights
        if (a.n_q_heads / a.n_kv_heads > 16) return launch<TensorShape<VT, IO, 32>>(a, sms, stream);
    return launch<TensorShape<VT, IO, 16>>(a, sms, stream);
}

cudaError_t launch_latent_tensor(const AttendArgs &a, int32_t vt, int32_t io, int32_t sms, cudaStream_t stream) {
    if (vt == KVX_BF16) return launch_heads<KVX_BF16, KVX_BF16>(a, sms, stream);
    if (vt == KVX_F16) return launch_heads<KVX_F16, KVX_F16>(a, sms, stream);
    return io == KVX_BF16 ? launch_heads<KVX_E4M3, KVX_BF16>(a, sms, stream) : launch_heads<KVX_E4M3, KVX_F16>(a, sms, stream);
}

}  // namespace kvx
