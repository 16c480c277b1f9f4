// kvx_cache_attend_shared over the prefixes that groups of requests share, on the tcgen05 tensor pipe: the kernel, instantiated
// per value type in kvx_shared_*.cu. The plan before it is in kvx_shared_plan.cuh, the launches and the join after it in kvx_shared.cu; each
// request's own positions go through the kernel of kvx_attend_planes.cuh.
//
// The queries of all members of a group that read one KV head are the rows of one matrix Q (members x query heads of a KV head), so
// a prefix is attention with many queries:
//   S = Q K^T, m' = max(m, S), P = 2^(S - m'), l' = l 2^(m - m') + sum P, O' = O 2^(m - m') + P V.
// A unit is up to 256 rows of one KV head. Its prefix is cut into tiles of 128 positions, and all units' tiles stand in one line of
// which each CTA takes an equal stretch, so the load is level whatever the groups; each CTA leaves for a unit one partial result
// (O, m, l) in the workspace.
//
// A CTA has two slots, each with 128 rows of scores and sums in TMEM (S: 128 columns, O: 128), four softmax warps, a thread a row, and a
// warp of its own that issues its products. With more than 128 rows the slots are the two halves of the rows and share each tile of keys and
// values; with fewer they are the same rows and take every other tile. The slots' softmaxes take turns, so that while one slot's scores
// go through the softmax the tensor pipe has the other's products; weights are handed over a quarter of a tile at a time. The
// weights go back into the columns of their scores as operand A, as two 16-bit values each, whose sum leaves 2^-16 of a weight (bf16)
// or 2^-20 (f16, or 2^-35 of the row's largest). An infinite value must meet neither a zero nor a negative value, which would make it NaN: the first is cut
// off, not rounded, and the second is never zero.
//
// Keys and values come row by row with asynchronous copies of 16 bytes, so pages of any size and layout will do, into rings
// whose rows of 64 elements are swizzled over 128 bytes: K-major for the scores, MN-major for the sums. Their arrival is the copies' own;
// the proxy fence stands where they are used (where they are made it had each copying thread wait for its copies). 8-bit codes pass through
// registers and become f16, which holds them exactly (1000 clocks of the copies' warps for a tile of keys or values).
//
// Bound by the tensor pipe where many rows share (with the weights' second value three products, not two): 64 requests on a document of 32768
// positions, 64 + 8 heads of 128, 68 us, 1.0 PFLOP/s of scores and sums, 1.5 with the second value, 0.79 of the measured rate; else by what a CTA's one
// or two units cost apart from their tiles (first keys 3 us, flush 2). Steps, of the same case (us): first form 129; a whole row of scores in
// registers (setmaxnreg) 113; arrivals without the copying threads, operands made uniform by __reduce_max_sync 85; a product warp for each slot, weights
// in halves 80; turns and quarters 68. Not kept: turns handed over earlier 68.5, stores of 16 columns 70, whole numbers of CTAs for each unit 73,
// the requests' own positions as units 127.
#pragma once

#include "kvx_shared_plan.cuh"
#include "kvx_tensor.cuh"

namespace kvx {

constexpr int kSharedThreads = 16 * 32;                            // warps 0-7: softmax, four a slot; 8, 9: products; 12-15: copies
constexpr int kSharedLoaders = 128;
constexpr int kSharedMin = 4;                                      // places of a CTA at least
constexpr float kSharedSlack = 3.0f;                               // by which a score may pass the maximum, in powers of two
constexpr uint32_t kSharedColSums = 0, kSharedColScores = 256;     // of TMEM: per slot 128

__device__ __forceinline__ int64_t part_bytes(int32_t head_dim) { return 2 * kSharedRows * ((int64_t)head_dim * 4 + 8); }

__device__ __forceinline__ Split shared_split(int64_t places, int ctas) {
    return Split{places, (int32_t)min((int64_t)ctas, divide(places + kSharedMin - 1, kSharedMin))};
}

// What a CTA has of a unit.
struct SharedWork {
    SharedUnit u;
    int32_t index;                     // of the unit
    int32_t t0, n;                     // tiles [t0, t0 + n)
    bool both;                         // both slots take each tile
    // To the next unit of the CTA's stretch from `index` on; false: none.
    __device__ __forceinline__ bool read(const SharedArgs &s, int64_t c_begin, int64_t c_end, int32_t units) {
        for (; index < units; ++index) {
            u = s.units[index];
            if (u.begin >= c_end) return false;
            const int w = shared_weight(u.rows);
            const int64_t places = (int64_t)shared_tiles(u.tokens) * w;
            const int64_t lo = max(c_begin, u.begin) - u.begin, hi = min(c_end, u.begin + places) - u.begin;
            if (hi <= lo) continue;
            both = w == 2;
            t0 = (int32_t)((lo + w - 1) >> (w - 1));
            n = (int32_t)((hi + w - 1) >> (w - 1)) - t0;
            return true;
        }
        return false;
    }
};

template <int VT_, int IO_, int D_> struct SharedShape {
    static constexpr int VT = VT_, IO = IO_, D = D_;               // D: head_dim rounded up to 64 or 128
    static constexpr bool F8 = VT == KVX_E4M3;
    static constexpr int MT = F8 ? KVX_F16 : VT;                   // type of the products
    static constexpr int CHUNKS = D / 64, CHUNK = kSharedTile * 128, TILE = CHUNKS * CHUNK;   // bytes; a chunk: 64 elements of 128 rows
    static constexpr int OFF_RING = 2 * TILE;                      // behind the queries of the two slots
    static constexpr int STAGES = ((224 << 10) - OFF_RING) / TILE < 8 ? ((224 << 10) - OFF_RING) / TILE : 8;
    static constexpr int BYTES = OFF_RING + STAGES * TILE;
    static constexpr float UP = MT == KVX_F16 ? 12.0f : 0.0f;      // f16 weights are taken times 2^12, up to 2^15: their step is 2^-36
    static constexpr uint32_t IDESC = 1u << 4 | (MT == KVX_BF16 ? 1u << 7 | 1u << 10 : 0) | (uint32_t)(kSharedRows / 16) << 24;
    static constexpr uint32_t IDESC_SCORES = IDESC | (uint32_t)(kSharedTile / 8) << 17;
    static constexpr uint32_t IDESC_SUMS = IDESC | (uint32_t)(D / 8) << 17 | 1u << 16;        // V by columns
    // Registers a thread: a softmax warp holds a row's 128 scores. Four warpgroups of 128 at the launch are 512.
    static constexpr int REGS_SOFTMAX = F8 ? 168 : 184, REGS_PRODUCTS = 64, REGS_COPIES = F8 ? 112 : 80;
    static_assert(2 * REGS_SOFTMAX + REGS_PRODUCTS + REGS_COPIES <= 512, "a warpgroup would wait for registers that nobody has");
    static constexpr int PIECES = D / 8;                           // of 16 bytes in a row of shared memory
    static_assert(STAGES >= 4, "keys and values of two tiles");
    static_assert(BYTES <= (224 << 10), "3 KiB are the barriers' and the slots' maxima and sums");
};

// The product with operand A in TMEM.
__device__ __forceinline__ void tensor_mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n.reg .pred p, e;\nsetp.ne.u32 p, %4, 0;\nelect.sync _|e, 0xffffffff;\n"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
                 : "memory");
}

// 32 columns of this warp's 32 rows of TMEM.
__device__ __forceinline__ void tmem_load32(uint32_t (&x)[32], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,"
        "%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]),
          "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]), "=r"(x[16]), "=r"(x[17]), "=r"(x[18]), "=r"(x[19]), "=r"(x[20]),
          "=r"(x[21]), "=r"(x[22]), "=r"(x[23]), "=r"(x[24]), "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]), "=r"(x[30]),
          "=r"(x[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_store32(const uint32_t (&x)[32], uint32_t at) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,"
        "%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
        "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]), "r"(x[10]), "r"(x[11]),
        "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]), "r"(x[16]), "r"(x[17]), "r"(x[18]), "r"(x[19]), "r"(x[20]), "r"(x[21]), "r"(x[22]),
        "r"(x[23]), "r"(x[24]), "r"(x[25]), "r"(x[26]), "r"(x[27]), "r"(x[28]), "r"(x[29]), "r"(x[30]), "r"(x[31])
        : "memory");
}

// Two values at a time.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\nfma.rn.f32x2 d, a, b, c;\nmov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Registers of this warpgroup's threads from here on; what the others give up.
template <int N> __device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void leave_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Two weights as two values each.
template <class S> __device__ __forceinline__ void two_values(float2 p, uint32_t &hi, uint32_t &lo) {
    if constexpr (S::MT == KVX_BF16) {                             // what is cut off, and 2^-23 of the rest: never zero
        const float2 minus = make_float2(-1.0f + 0x1p-23f, -1.0f + 0x1p-23f);
        hi = __byte_perm(__float_as_uint(p.x), __float_as_uint(p.y), 0x7632);
        const float2 top = make_float2(__uint_as_float(__float_as_uint(p.x) & 0xffff0000u), __uint_as_float(__float_as_uint(p.y) & 0xffff0000u));
        const float2 rest = fma2(top, minus, p);
        lo = pack<KVX_BF16>(rest.x, rest.y);
    } else if constexpr (S::F8) {                                  // 8-bit values are finite
        const float2 minus = make_float2(-1.0f, -1.0f);
        hi = pack<KVX_F16>(p.x, p.y);
        const float2 rest = fma2(unpack<KVX_F16>(hi), minus, p);
        lo = pack<KVX_F16>(rest.x, rest.y);
    } else {
        const float2 minus = make_float2(-1.0f, -1.0f);
        hi = pack_down<KVX_F16>(p.x, p.y);
        const float2 rest = fma2(unpack<KVX_F16>(hi), minus, p);
        lo = pack_down<KVX_F16>(rest.x, rest.y) | 0x00010001u;     // cut off to an odd last place
    }
}

// This thread's copies so far count as an arrival once they are through.
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(shared_addr(bar)) : "memory");
}

template <class S> __global__ void __launch_bounds__(kSharedThreads, 1) kvx_attend_shared(const __grid_constant__ SharedArgs s) {
    extern __shared__ __align__(1024) uint8_t smem[];              // queries of the slots, then the ring
    __shared__ __align__(8) uint64_t s_full[S::STAGES], s_free[S::STAGES], s_queried, s_unqueried;
    __shared__ __align__(8) uint64_t s_scored[2], s_weighed[2][4], s_summed[2], s_turn[2], s_drained[2], s_never;   // per slot; weights in quarters of a tile
    __shared__ __align__(8) uint64_t s_met, s_left;                // both slots' sums of a unit are there; the second slot has read them
    __shared__ float2 s_ml[2][kSharedRows];                        // of slots that share their rows
    __shared__ __align__(16) uint32_t s_live[8][4];                // live positions of the last tiles
    __shared__ int8_t s_up[2][2][S::F8 ? kSharedRows : 1];         // by turns of units, per slot: powers of two of 8-bit caches' bf16 queries
    __shared__ uint32_t s_tmem;
    __shared__ int32_t s_first;
    __shared__ volatile int32_t s_failed;
    const AttendArgs &a = s.a;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {                                        // what touches no memory, while the kernel before still runs
        s_failed = 0;
        auto init = [](uint64_t *bar, int n) { asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_addr(bar)), "r"(n) : "memory"); };
        for (int i = 0; i < S::STAGES; ++i) {
            init(&s_full[i], S::F8 ? kSharedLoaders : kSharedLoaders + 4);
            init(&s_free[i], 2);                                   // each slot's products, or twice those of the one that took it
        }
        for (int i = 0; i < 2; ++i) {
            init(&s_scored[i], 1);
            for (int h = 0; h < 4; ++h) init(&s_weighed[i][h], kSharedRows);
            init(&s_summed[i], 1);
            init(&s_turn[i], kSharedRows);
            init(&s_drained[i], 1);
        }
        init(&s_queried, kSharedLoaders);
        init(&s_unqueried, 2);
        init(&s_never, 1);
        init(&s_met, 2 * kSharedRows);
        init(&s_left, kSharedRows);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    wait_for_earlier();
    const int64_t places = s.header->places;
    const int32_t units = s.header->units;
    const Split split = shared_split(places, gridDim.x);
    if (places == 0 || (int32_t)blockIdx.x >= split.ctas) return;
    const int64_t c_begin = split.begin(blockIdx.x), c_end = split.begin(blockIdx.x + 1);
    if (w == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_addr(&s_tmem)), "n"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tensor_fence_before();
    }
    if (w == 0) {                                                  // the unit that holds c_begin
        int32_t lo = 0, n = units;
        while (n > 1) {
            const int32_t step = (n + 31) / 32, at = lane * step;
            const uint32_t upto = __ballot_sync(~0u, at < n && s.units[lo + at].begin <= c_begin);
            const int32_t k = (31 - __clz(upto)) * step;
            lo += k;
            n = min(step, n - k);
        }
        if (lane == 0) s_first = lo;
    }
    __syncthreads();
    tensor_fence_after();
    const uint32_t tmem = s_tmem;
    // Of any role, by a whole warp: false when it, or another role's, ran out. All lanes have the same answer, as they take part in what
    // follows together (instructions on TMEM): one lane could see a phase that has come just as another one's wait runs out.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (__all_sync(~0u, phase_done(bar, parity & 1))) return true;
        const bool ok = __all_sync(~0u, !s_failed && wait_full(bar, parity & 1, a.wait_ns));
        if (!ok) s_failed = 1;
        return ok;
    };
    auto goes_on = [&](int part) { return a.stall != part || blockIdx.x != 0 || wait(&s_never, 0); };   // the testing hook
    const int32_t group = a.n_q_heads / a.n_kv_heads;
    SharedWork work;
    work.index = s_first;

    if (w < 8) {                                                   // softmax and partial results
        take_registers<S::REGS_SOFTMAX>();
        const int slot = w >> 2, row = (w & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(w & 3) << 21);
        const uint32_t sums = lanes + kSharedColSums + slot * 128, scores = lanes + kSharedColScores + slot * 128;
        int tiles = 0, scored = 0, summed = 0, turn = 0, round = 0, met = 0;   // tiles of the units before; phases; units with tiles; turns
        bool ok = goes_on(kStallSharedSoftmax);
        for (; ok && work.read(s, c_begin, c_end, units); ++work.index) {
            const int steps = work.both ? work.n : (work.n + 1 - slot) / 2, rounds = work.both ? work.n : (work.n + 1) / 2;
            float m = -INFINITY, sc = a.scale;                     // m: of the scores, less UP
            float2 l = make_float2(0.0f, 0.0f);
            for (int i = 0; i < rounds; ++i, ++round) {
                // The slots' softmaxes take turns: alone one takes half as long, and the pipe has the other's products meanwhile.
                if (i < steps && !(ok = wait(&s_scored[slot], scored++))) break;
                if ((slot || round) && !(ok = wait(&s_turn[slot], slot ? round : round - 1))) break;
                if (i >= steps) {
                    arrive(&s_turn[slot ^ 1]);
                    continue;
                }
                tensor_fence_after();
                if constexpr (S::F8 && S::IO == KVX_BF16)
                    if (i == 0) sc = fmaxf(a.scale * __int_as_float((127 - s_up[turn & 1][work.both ? slot : 0][row]) << 23), kLeastScale);
                const uint4 four = *reinterpret_cast<const uint4 *>(s_live[(tiles + (work.both ? i : 2 * i + slot)) & 7]);
                const uint32_t live[4] = {four.x, four.y, four.z, four.w};
                const bool all = (four.x & four.y & four.z & four.w) == ~0u;
                uint32_t x[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_load32(x[c], scores + c * 32);
                tmem_load_wait();
                if (!all) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(live[c] >> k & 1)) x[c][k] = 0xff800000u;            // -infinity
                }
                float y[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 32; k += 2)
#pragma unroll
                    for (int c = 0; c < 4; ++c) y[c] = max3(y[c], __uint_as_float(x[c][k]), __uint_as_float(x[c][k + 1]));
                const float top = fmaf(max3(fmaxf(y[0], y[1]), y[2], y[3]), sc, -S::UP);
                const bool moves = top > m + kSharedSlack;
                if (__any_sync(~0u, moves)) {                      // the products of this slot's tile before are done: these scores came after
                    const float up = moves ? top : m, old = moves ? fast_exp2(m - up) : 1.0f;
                    m = up;
                    l.x *= old;
                    l.y *= old;
                    if (i > 0)
#pragma unroll 1
                        for (int c = 0; c < S::D; c += 8) {
                            uint32_t o[8];
                            tmem_load(o, sums + c);
                            tmem_load_wait();
#pragma unroll
                            for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * old);
                            tmem_store(o, sums + c);
                        }
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                const float2 sc2 = make_float2(sc, sc), ref2 = make_float2(-ref, -ref);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t z[32];                                // the first values of 32 weights, then the second ones
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 e = fma2(make_float2(__uint_as_float(x[c][2 * k]), __uint_as_float(x[c][2 * k + 1])), sc2, ref2);
                        const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));
                        l = add2(l, p);
                        two_values<S>(p, z[k], z[16 + k]);
                    }
                    if (c) {                                       // the quarter before is stored by now: its products begin
                        tmem_store_wait();
                        tensor_fence_before();
                        arrive(&s_weighed[slot][c - 1]);
                    }
                    tmem_store32(z, scores + c * 32);
                }
                arrive(&s_turn[slot ^ 1]);
                tmem_store_wait();
                tensor_fence_before();
                arrive(&s_weighed[slot][3]);
            }
            if (!ok) break;
            // the partial result
            const bool real = (work.both ? slot * kSharedRows : 0) + row < work.u.rows;
            uint8_t *const part = s.parts + (int64_t)(work.index + blockIdx.x) * part_bytes(a.head_dim) + (work.both ? slot * (part_bytes(a.head_dim) / 2) : 0);
            float4 *const to = reinterpret_cast<float4 *>(part + kSharedRows * 8) + row;
            const float2 mine = make_float2(m, l.x + l.y);
            if (steps && !(ok = wait(&s_summed[slot], summed++))) break;
            tensor_fence_after();
            if (!work.both) {                                      // of the same rows: joined here, half of the columns by each slot
                s_ml[slot][row] = mine;
                tensor_fence_before();
                arrive(&s_met);
                if (!(ok = wait(&s_met, met))) break;
                tensor_fence_after();
                const float2 one = s_ml[0][row], two = s_ml[1][row];
                const float up = fmaxf(one.y != 0.0f ? one.x : -INFINITY, two.y != 0.0f ? two.x : -INFINITY), ref = up == -INFINITY ? 0.0f : up;
                const float by_one = one.y != 0.0f ? fast_exp2(one.x - ref) : 0.0f, by_two = two.y != 0.0f ? fast_exp2(two.x - ref) : 0.0f;
                if (slot == 0 && real) __stcg(reinterpret_cast<float2 *>(part) + row, make_float2(up, fmaf(one.y, by_one, two.y * by_two)));
#pragma unroll 1
                for (int c = slot * (S::D / 2); c < (slot + 1) * (S::D / 2); c += 32) {
                    uint32_t o[2][32];
                    tmem_load32(o[0], lanes + kSharedColSums + c);
                    tmem_load32(o[1], lanes + kSharedColSums + 128 + c);
                    tmem_load_wait();
                    float z[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {                 // sums without weights may be anything
                        const float p = one.y != 0.0f ? __uint_as_float(o[0][k]) * by_one : 0.0f;
                        z[k] = two.y != 0.0f ? fmaf(__uint_as_float(o[1][k]), by_two, p) : p;
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (real && c + 4 * k < a.head_dim)
                            __stcg(to + (c / 4 + k) * kSharedRows, make_float4(z[4 * k], z[4 * k + 1], z[4 * k + 2], z[4 * k + 3]));
                }
                tensor_fence_before();
                // The second slot's next products come after the first one's next softmax, which comes after this.
                if (slot) arrive(&s_left);
                else if (!(ok = wait(&s_left, met))) break;
                ++met;
            } else if (steps) {
                if (real) __stcg(reinterpret_cast<float2 *>(part) + row, mine);
#pragma unroll 1
                for (int c = 0; c < S::D; c += 32) {
                    uint32_t o[32];
                    tmem_load32(o, sums + c);
                    tmem_load_wait();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (real && c + 4 * k < a.head_dim)
                            __stcg(to + (c / 4 + k) * kSharedRows, make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                                                               __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3])));
                }
                tensor_fence_before();
            } else if (real) __stcg(reinterpret_cast<float2 *>(part) + row, mine);
            tiles += work.n;
            turn += work.n > 0;
        }
    } else if (w < 12) {                                           // products, of a slot by each of the first two of these warps
        leave_registers<S::REGS_PRODUCTS>();
        // A slot's products are issued in their order by one warp and go through the pipe in it, so that the scores of its next tile
        // may take the place of the weights as soon as they are issued. What the operands are made of is the same in all lanes;
        // it comes from reductions, so that the compiler knows it too.
        const int slot = (int)__reduce_max_sync(~0u, (uint32_t)(w - 8));
        const uint32_t columns = __reduce_max_sync(~0u, tmem);
        const uint64_t queries = operand(shared_addr(smem), 16, 1024, 2), ring = operand(shared_addr(smem + S::OFF_RING), 16, 1024, 2);
        const uint64_t values = operand(shared_addr(smem + S::OFF_RING), S::CHUNK, 1024, 2);
        const uint32_t scores = columns + kSharedColScores + slot * 128, sums = columns + kSharedColSums + slot * 128;
        int item = 0, turn = 0, weighed = 0;
        bool ok = slot < 2 && goes_on(kStallSharedProducts);
        for (; ok && work.read(s, c_begin, c_end, units); ++work.index) {
            const int n = (int)__reduce_max_sync(~0u, (uint32_t)work.n);
            if (n == 0) continue;
            const bool both = __any_sync(~0u, work.both);
            const int first = both ? 0 : slot, step = both ? 1 : 2;            // the slot's tiles
            if (!(ok = wait(&s_queried, turn++))) break;
            fence_async();                                         // copies come by the generic proxy, products read by the other
            const uint64_t q = queries + (both ? slot * (S::TILE / 16) : 0);
            auto release = [&](int stage) {
                tensor_commit(&s_free[stage]);
                if (!both) tensor_commit(&s_free[stage]);
            };
            auto key_stage = [&](int t) { return t ? item + 2 * t - 1 : item; };
            auto copied = [&](int at) {
                ok = ok && wait(&s_full[at % S::STAGES], at / S::STAGES);
                fence_async();
            };
            auto score = [&](int t) {
                const int stage = key_stage(t) % S::STAGES;
                const uint64_t keys = ring + stage * (S::TILE / 16);
#pragma unroll
                for (int y = 0; y < S::D / 16; ++y)                // 32 bytes of the rows
                    tensor_mma<false>(scores, q + y / 4 * (S::CHUNK / 16) + y % 4 * 2, keys + y / 4 * (S::CHUNK / 16) + y % 4 * 2, S::IDESC_SCORES, y > 0);
                tensor_commit(&s_scored[slot]);
                release(stage);
                if (t + step >= n) tensor_commit(&s_unqueried);
            };
            if (first < n) {
                copied(key_stage(first));
                if (!ok) break;
                score(first);
            } else tensor_commit(&s_unqueried);
            for (int t = first; ok && t < n; t += step, ++weighed) {
                const int at = t + 1 < n ? item + 2 * t + 2 : item + 2 * n - 1;
                const bool more = t + step < n;
                copied(at);                                        // while the softmax is at work
                const uint64_t v = values + at % S::STAGES * (S::TILE / 16);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    ok = ok && wait(&s_weighed[slot][h], weighed);
                    if (!ok) break;
                    tensor_fence_after();
#pragma unroll
                    for (int y = 2 * h; y < 2 * h + 2; ++y)        // 16 positions
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            tensor_mma_tmem(sums, scores + y / 2 * 32 + i * 16 + y % 2 * 8, v + y * (2048 / 16), S::IDESC_SUMS, t != first || y > 0 || i > 0);
                    if (h == 2 && more) copied(key_stage(t + step));
                }
                if (!ok) break;
                if (more) score(t + step);
                release(at % S::STAGES);
                if (!more) tensor_commit(&s_summed[slot]);
            }
            item += 2 * n;
        }
    } else {                                                       // copies
        leave_registers<S::REGS_COPIES>();
        const int lw = w - 12;
        int item = 0, turn = 0, tiles = 0;
        bool ok = goes_on(kStallSharedCopies);
        const uint32_t smem0 = shared_addr(smem);
        // Position `lane` of this warp's quarter of a tile: its block, -2 behind the prefix; then its row's offset in its buffer, in
        // 16-byte units. In two steps, so that the block's id is on its way a tile ahead.
        auto block_of = [&](int tile) {
            const uint32_t pos = (uint32_t)tile * kSharedTile + lw * 32 + lane;
            if (pos >= (uint32_t)work.u.tokens) return -2;
            return max(a.block_table[work.u.first * a.table_stride + ((__umulhi(pos, a.block_mul) + pos) >> a.block_shift)], -1);
        };
        auto row_of = [&](int32_t blk, int tile) {
            const uint32_t pos = (uint32_t)tile * kSharedTile + lw * 32 + lane, col = (__umulhi(pos, a.block_mul) + pos) >> a.block_shift;
            uint32_t at = kNoRow;
            if (blk >= 0 && blk < a.pool.n_blocks) at = (uint32_t)blk * a.block_pitch16 + (pos - col * (uint32_t)a.pool.block_size) * a.token_pitch16;
            else if (blk != -2 && work.u.kvh == 0 && work.u.pair == 0) atomicAdd(a.pool.skipped, 1ull);
            return at;
        };
        auto set_live = [&](int tile, uint32_t row) {
            const uint32_t bits = __ballot_sync(~0u, row != kNoRow);
            if (lane == 0) s_live[tile & 7][lw] = bits;
        };
        auto query_row = [&](int r) {                              // of the unit; NULL: none
            if (r >= work.u.rows) return (const uint8_t *)nullptr;
            const uint32_t at = (uint32_t)(work.u.pair * 2 * kSharedRows + r), member = at / (uint32_t)group;
            return a.q + (int64_t)(work.u.first + (int32_t)member) * a.q_stride +
                   ((int64_t)work.u.kvh * group + (at - member * (uint32_t)group)) * a.head_dim * 2;
        };
        if constexpr (!S::F8) {
            constexpr int AT_ONCE = 32 / S::PIECES;                // rows that a copy of the warp covers
            const int piece = lane % S::PIECES;
            const bool piece_in = piece * 8 < a.head_dim;
            const uint32_t piece_at = piece / 8 * S::CHUNK;
            auto place = [&](int r) { return piece_at + r * 128 + ((piece % 8) ^ (r & 7)) * 16; };
            auto put = [&](const uint8_t *from, uint32_t row) {
                if (item >= S::STAGES) ok = ok && wait(&s_free[item % S::STAGES], item / S::STAGES - 1);
                if (!ok) return;
                const uint32_t to = smem0 + S::OFF_RING + item % S::STAGES * S::TILE;
                from += piece * 16;
#pragma unroll
                for (int i = 0; i < S::PIECES; ++i) {
                    const int r = i * AT_ONCE + lane / S::PIECES;
                    const uint32_t at = __shfl_sync(~0u, row, r);
                    const bool in = at != kNoRow && piece_in;
                    copy_async(to + place(lw * 32 + r), from + (in ? (uint64_t)at * 16 : 0), in);
                }
                copies_arrive(&s_full[item % S::STAGES]);
                if (lane == 0) arrive(&s_full[item % S::STAGES]);     // with what it wrote to s_live
                ++item;
            };
            for (; ok && work.read(s, c_begin, c_end, units); ++work.index) {
                if (work.n == 0) continue;
                const int32_t shard = work.u.kvh / a.pool.heads_per_shard;
                const int64_t head = (int64_t)(work.u.kvh - shard * a.pool.heads_per_shard) * a.pool.head_pitch;
                const uint8_t *const keys = a.pool.k[shard] + head, *const vals = a.pool.v[shard] + head;
                // keys of a tile, then values of the one before
                uint32_t row = row_of(block_of(work.t0), work.t0), next = row;
                int32_t blk = work.n > 1 ? block_of(work.t0 + 1) : -2;
                set_live(tiles, row);
                put(keys, row);
                for (int t = 0; ok && t < work.n; ++t) {
                    if (t + 1 < work.n) {
                        next = row_of(blk, work.t0 + t + 1);
                        if (t + 2 < work.n) blk = block_of(work.t0 + t + 2);
                        set_live(tiles + t + 1, next);
                        put(keys, next);
                    }
                    if (!ok) break;
                    put(vals, row);
                    row = next;
                    if (t) continue;
                    // Queries, once those before have been multiplied.
                    if (turn) ok = ok && wait(&s_unqueried, turn - 1);
                    if (!ok) break;
                    for (int b = 0; b < (work.both ? 2 : 1); ++b) {
                        const uint64_t mine = (uint64_t)query_row(b * kSharedRows + lw * 32 + lane);
#pragma unroll
                        for (int i = 0; i < S::PIECES; ++i) {
                            const int r = i * AT_ONCE + lane / S::PIECES;
                            const uint64_t p = __shfl_sync(~0u, mine, r);
                            const bool in = p != 0 && piece_in;
                            copy_async(smem0 + b * S::TILE + place(lw * 32 + r), in ? (const uint8_t *)p + piece * 16 : a.q, in);
                        }
                    }
                    copies_arrive(&s_queried);
                    ++turn;
                }
                tiles += work.n;
            }
            copies_commit();
            copies_wait<0>();                                      // none outlives the CTA
        } else {
            // A row has D / 16 pieces of 16 codes; a lane reads READS of its warp's 32 rows.
            constexpr int CODES = S::D / 16, READS = CODES, AT_ONCE = 32 / CODES;
            const int piece = lane % CODES;
            const bool piece_in = piece * 16 < a.head_dim;
            uint4 x[2][READS];
            auto fetch = [&](uint4 (&y)[READS], const uint8_t *from, uint32_t row) {
#pragma unroll
                for (int i = 0; i < READS; ++i) {
                    const uint32_t at = __shfl_sync(~0u, row, i * AT_ONCE + lane / CODES);
                    y[i] = at != kNoRow && piece_in ? __ldg(reinterpret_cast<const uint4 *>(from + (uint64_t)at * 16) + piece) : make_uint4(0, 0, 0, 0);
                }
            };
            // Two pieces of 8 elements beside one another.
            auto place = [&](uint32_t base, int r, int p) { return base + p / 8 * S::CHUNK + r * 128 + ((p % 8) ^ (r & 7)) * 16; };
            auto read = [&](uint32_t at) {
                uint4 y;
                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w) : "r"(at) : "memory");
                return y;
            };
            auto write = [&](uint32_t at, uint32_t y0, uint32_t y1, uint32_t y2, uint32_t y3) {
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(y0), "r"(y1), "r"(y2), "r"(y3) : "memory");
            };
            auto store = [&](const uint4 (&y)[READS]) {
                if (item >= S::STAGES) ok = ok && wait(&s_free[item % S::STAGES], item / S::STAGES - 1);
                if (!ok) return;
                const uint32_t to = smem0 + S::OFF_RING + item % S::STAGES * S::TILE;
#pragma unroll
                for (int i = 0; i < READS; ++i) {
                    const int r = lw * 32 + i * AT_ONCE + lane / CODES;
                    uint32_t z[8];
                    f16_of_codes(y[i].x, z[0], z[1]);
                    f16_of_codes(y[i].y, z[2], z[3]);
                    f16_of_codes(y[i].z, z[4], z[5]);
                    f16_of_codes(y[i].w, z[6], z[7]);
                    write(place(to, r, 2 * piece), z[0], z[1], z[2], z[3]);
                    write(place(to, r, 2 * piece + 1), z[4], z[5], z[6], z[7]);
                }
                arrive(&s_full[item % S::STAGES]);
                ++item;
            };
            // Queries as f16: a bf16 row is brought by a power of two to where f16 holds its elements exactly down to 2^-31 of the largest.
            // All rows are on their way at once, to the places where the lane that copied them turns them into f16.
            auto load_queries = [&]() {
                if (turn) ok = ok && wait(&s_unqueried, turn - 1);
                if (!ok) return;
                constexpr int LANES = S::PIECES, ROWS = 32 / LANES;
                const int p = lane % LANES, slots = work.both ? 2 : 1;
                for (int b = 0; b < slots; ++b) {
                    const uint64_t mine = (uint64_t)query_row(b * kSharedRows + lw * 32 + lane);
#pragma unroll
                    for (int i = 0; i < LANES; ++i) {
                        const int r = i * ROWS + lane / LANES;
                        const uint64_t src = __shfl_sync(~0u, mine, r);
                        const bool in = src != 0 && p * 8 < a.head_dim;
                        copy_async(place(smem0 + b * S::TILE, lw * 32 + r, p), in ? (const uint8_t *)src + p * 16 : a.q, in);
                    }
                }
                copies_commit();
                copies_wait<0>();
                if constexpr (S::IO == KVX_BF16) {
                    constexpr int BATCH = 4;                           // whose chains of maxima overlap
                    for (int b = 0; b < slots; ++b) {
                        for (int i = 0; i < LANES; i += BATCH) {
                            uint4 y[BATCH];
                            float top[BATCH];
#pragma unroll
                            for (int k = 0; k < BATCH; ++k) {
                                y[k] = read(place(smem0 + b * S::TILE, lw * 32 + (i + k) * ROWS + lane / LANES, p));
                                const float2 f[4] = {unpack<KVX_BF16>(y[k].x), unpack<KVX_BF16>(y[k].y), unpack<KVX_BF16>(y[k].z), unpack<KVX_BF16>(y[k].w)};
                                top[k] = 0.0f;
#pragma unroll
                                for (int j = 0; j < 4; ++j) top[k] = fmaxf(top[k], fmaxf(fabsf(f[j].x), fabsf(f[j].y)));
                            }
#pragma unroll
                            for (int d = 1; d < LANES; d <<= 1)
#pragma unroll
                                for (int k = 0; k < BATCH; ++k) top[k] = fmaxf(top[k], __shfl_xor_sync(~0u, top[k], d));
#pragma unroll
                            for (int k = 0; k < BATCH; ++k) {
                                const int r = lw * 32 + (i + k) * ROWS + lane / LANES;
                                const float2 f[4] = {unpack<KVX_BF16>(y[k].x), unpack<KVX_BF16>(y[k].y), unpack<KVX_BF16>(y[k].z), unpack<KVX_BF16>(y[k].w)};
                                const int exponent = (__float_as_int(top[k]) >> 23) - 127;         // of numbers below the smallest normal one -127
                                const int e = top[k] > 0.0f && top[k] < INFINITY ? max(-126, min(100, 14 - exponent)) : 0;
                                const float up = __int_as_float((127 + e) << 23);
                                write(place(smem0 + b * S::TILE, r, p), pack<KVX_F16>(f[0].x * up, f[0].y * up), pack<KVX_F16>(f[1].x * up, f[1].y * up),
                                      pack<KVX_F16>(f[2].x * up, f[2].y * up), pack<KVX_F16>(f[3].x * up, f[3].y * up));
                                if (p == 0) s_up[turn & 1][b][r] = (int8_t)e;
                            }
                        }
                    }
                }
                arrive(&s_queried);
                ++turn;
            };
            for (; ok && work.read(s, c_begin, c_end, units); ++work.index) {
                if (work.n == 0) continue;
                const int32_t shard = work.u.kvh / a.pool.heads_per_shard;
                const int64_t head = (int64_t)(work.u.kvh - shard * a.pool.heads_per_shard) * a.pool.head_pitch;
                const uint8_t *const keys = a.pool.k[shard] + head, *const vals = a.pool.v[shard] + head;
                // keys of tile t + 1, then values of tile t: each read while the one before is written
                uint32_t row = row_of(block_of(work.t0), work.t0), next = row;
                int32_t blk = work.n > 1 ? block_of(work.t0 + 1) : -2;
                fetch(x[0], keys, row);
                set_live(tiles, row);
                load_queries();
                if (ok) store(x[0]);
                if (work.n > 1) {
                    next = row_of(blk, work.t0 + 1);
                    if (work.n > 2) blk = block_of(work.t0 + 2);
                    fetch(x[0], keys, next);
                }
                for (int t = 0; ok && t < work.n; ++t) {
                    fetch(x[1], vals, row);
                    if (t + 1 < work.n) {
                        set_live(tiles + t + 1, next);
                        store(x[0]);
                        row = next;
                    }
                    if (t + 2 < work.n) {
                        next = row_of(blk, work.t0 + t + 2);
                        if (t + 3 < work.n) blk = block_of(work.t0 + t + 3);
                        fetch(x[0], keys, next);
                    }
                    if (ok) store(x[1]);
                }
                tiles += work.n;
            }
        }
    }
    tensor_fence_before();
    __syncthreads();
    if (s_failed) {                                                // no product outlives the CTA, whoever's wait ran out
        if (w == 8 || w == 9) {
            tensor_commit(&s_drained[w - 8]);
            wait_full(&s_drained[w - 8], 0, kCacheWaitNs);
        }
        tensor_fence_before();
        __syncthreads();
    }
    if (w == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
    if (threadIdx.x == 0 && s_failed) atomicAdd(a.pool.skipped + 1, 1ull);
}

template <class S> static cudaError_t launch_shared_shape(const SharedArgs &s, int32_t sms, cudaStream_t stream) {
    static std::atomic<uint64_t> asked;
    const cudaError_t e = allow_shared(kvx_attend_shared<S>, S::BYTES, s.a.device, asked);
    return e != cudaSuccess ? e : launch_after(kvx_attend_shared<S>, dim3(sms), kSharedThreads, S::BYTES, stream, s);
}

template <int VT, int IO> static cudaError_t launch_shared_type(const SharedArgs &s, int32_t sms, cudaStream_t stream) {
    return s.a.head_dim <= 64 ? launch_shared_shape<SharedShape<VT, IO, 64>>(s, sms, stream) : launch_shared_shape<SharedShape<VT, IO, 128>>(s, sms, stream);
}

}  // namespace kvx
