// What the attention kernels share: the warp matrix product, conversions, and the split of a batch's work
// over the CTAs.
#pragma once

#include "kvx_launch.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace kvx {

constexpr uint32_t kNoRow = 0xffffffffu;      // offset of a position that is left out
constexpr float kLn2 = 0.6931471805599453f;

// D += A B, 16 x 8 x 16, 32-bit sums. bf16 values for KVX_BF16, else f16.
template <int VT>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (VT == KVX_BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit elements held by the warp, two of a row per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The four f16 values that a register of 8-bit codes stands for (exact).
__device__ __forceinline__ void f16_of_codes(uint32_t x, uint32_t &lo, uint32_t &hi) {
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}" : "=r"(lo), "=r"(hi) : "r"(x));
}

template <int VT> __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t y;
    if constexpr (VT == KVX_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}

// The same, cut off instead of rounded.
template <int VT> __device__ __forceinline__ uint32_t pack_down(float lo, float hi) {
    uint32_t y;
    if constexpr (VT == KVX_BF16) asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    else asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}

template <int VT> __device__ __forceinline__ float2 unpack(uint32_t x) {
    if constexpr (VT == KVX_BF16) return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Copies 16 bytes of the cache to shared memory in the background, zeros where the position is left out.
__device__ __forceinline__ void copy_async(uint32_t to, const uint8_t *p, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(p), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void shared_read(uint32_t (&x)[4], uint32_t at) {
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void shared_read(uint32_t (&x)[2], uint32_t at) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(at) : "memory");
}

// ------------------------------------------------------------------------------------------------
// The split of a batch. A segment is what one softmax runs over for one set of query heads: (request,
// head set); its positions are cut into tiles. All segments' tiles stand in one line, requests in order,
// and each CTA takes an equal stretch of it, so the load is level whatever the lengths. A segment that
// crosses from one CTA to the next is joined from the CTAs' partial sums in the scratch by whichever CTA
// finishes last, in the order of the line, so the result does not depend on which that is.
// ------------------------------------------------------------------------------------------------

// x / d, in 32 bits where they suffice.
__device__ __forceinline__ int64_t divide(int64_t x, int64_t d) {
    return (uint64_t)(x | d) >> 32 ? x / d : (int64_t)((uint32_t)x / (uint32_t)d);
}

// In proportion, not in whole tiles each: where the segments are alike and divide the CTAs, no CTA has parts of two.
struct Split {
    int64_t tiles;        // in all
    int32_t ctas;         // that have work, at least one tile each
    __device__ __forceinline__ int64_t begin(int32_t cta) const { return divide(cta * tiles, ctas); }
    __device__ __forceinline__ int32_t cta_of(int64_t tile) const { return (int32_t)divide((tile + 1) * ctas - 1, tiles); }
};

// A request's live positions [first, len) and its tiles of TOK positions, aligned to TOK; at least one, so that an
// empty request is answered too.
template <int TOK> struct Span {
    int32_t len, first, tiles;
    __device__ __forceinline__ Span(const AttendArgs &a, int32_t r) {
        const int64_t cap = (int64_t)a.max_blocks * a.pool.block_size;
        len = (int32_t)min((int64_t)max(a.seq_len[r], 0), cap);
        first = a.window ? max(0, len - a.window) : 0;
        tiles = max(1, (int32_t)(((uint32_t)len + TOK - 1) / TOK) - first / TOK);
    }
};

// Where a tile stands in the line. A segment has EXTRA places after its tiles, for what the change to the next one costs: they
// make the stretches even in time.
template <int TOK, int EXTRA> struct Place {
    int32_t r, seg, tile;      // request, segment of the request, tile of the segment
    int64_t before;            // places of the requests before r, per segment
    int32_t len, first, tiles;
    __device__ __forceinline__ void request(const AttendArgs &a) {
        const Span<TOK> s(a, r);
        len = s.len;
        first = s.first;
        tiles = s.tiles;
    }
    // To the next tile, and x with it.
    __device__ __forceinline__ void next(const AttendArgs &a, int32_t segs, int64_t &x) {
        ++x;
        if (++tile < tiles) return;
        x += EXTRA;
        tile = 0;
        if (++seg < segs) return;
        seg = 0;
        before += tiles + EXTRA;
        if (++r < a.n_reqs) request(a);
    }
    __device__ __forceinline__ int64_t seg_begin(int32_t segs) const { return before * segs + (int64_t)seg * (tiles + EXTRA); }
};

__device__ __forceinline__ int64_t warp_inclusive(int64_t x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x += o;
    }
    return x;
}

// Exclusive sum over the CTA's threads and the total.
template <int WARPS> __device__ __forceinline__ int64_t cta_exclusive(int64_t x, int64_t *total) {
    __shared__ int64_t sums[WARPS];
    const int64_t s = warp_inclusive(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 31) sums[threadIdx.x >> 5] = s;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        if (i == (int)(threadIdx.x >> 5)) before = all;
        all += sums[i];
    }
    *total = all;
    return before + s - x;
}

constexpr int kJoinTiles = 600;    // see Batch

// The batch as a CTA sees it: the split over gridDim.x CTAs (of at least MIN tiles each), and how to find a place in it.
// Where one CTA joins a segment's pieces, PIECES at a time, and there are few segments, not all CTAs get work: a segment of up
// to kJoinTiles tiles (on the average) goes to PIECES of them, one of up to k^2 kJoinTiles to k PIECES, so that the join takes as
// long as a stretch. One request on one KV head of 16384 bf16 positions 15.0 us, 22.1 on all CTAs; 32768 18.9, 25.7; 131072
// 31.7, 38.5. PIECES 0: always all CTAs.
// Up to 256 requests each warp keeps all the sums, a lane those of up to 8 consecutive requests, with no barrier; beyond that
// the CTA looks for the request in which its own stretch begins, and its warps go on from there.
template <int TOK, int WARPS, int MIN, int EXTRA, int PIECES> struct Batch {
    static constexpr int PER = 8;
    Split split;
    int32_t per;                       // requests of a lane
    int32_t tiles[PER];                // of each of them
    int64_t upto;                      // tiles of this lane's requests and those before
    int32_t r0;                        // beyond 256 requests: at or before this CTA's stretch, and the tiles before it
    int64_t before0;

    __device__ __forceinline__ Batch(const AttendArgs &a, int32_t segs) {
        const int lane = threadIdx.x & 31;
        const int64_t cap = (int64_t)a.max_blocks * a.pool.block_size;
        int64_t total = 0;
        per = (a.n_reqs + 31) / 32;
        if (per <= PER) {
            tiles[0] = lane * per < a.n_reqs ? Span<TOK>(a, lane * per).tiles + EXTRA : 0;
            int64_t mine = tiles[0];
#pragma unroll
            for (int k = 1; k < PER; ++k) tiles[k] = 0;
            if (per > 1)                   // else there are 32 requests at most, and a small call is spared the rest
#pragma unroll
                for (int k = 1; k < PER; ++k) {
                    const int32_t r = lane * per + k;
                    if (k < per && r < a.n_reqs) tiles[k] = Span<TOK>(a, r).tiles + EXTRA;
                    mine += tiles[k];
                }
            upto = warp_inclusive(mine);
            total = __shfl_sync(~0u, upto, 31);
        } else {
            int64_t mine = 0;
            for (int32_t r = threadIdx.x; r < a.n_reqs; r += 32 * WARPS) mine += Span<TOK>(a, r).tiles + EXTRA;
            cta_exclusive<WARPS>(mine, &total);
        }
        split.tiles = total * segs;
        split.ctas = (int32_t)min((int64_t)gridDim.x, divide(split.tiles + MIN - 1, MIN));
        if constexpr (PIECES > 0) {
            const int64_t segments = (int64_t)a.n_reqs * segs;
            for (int64_t k = 1; PIECES * k * segments < split.ctas; ++k)
                if (k * k * kJoinTiles * segments >= split.tiles) split.ctas = (int32_t)(PIECES * k * segments);
        }
        if (blockIdx.x == 0)
            for (int32_t r = threadIdx.x; r < a.n_reqs; r += 32 * WARPS)
                if (a.seq_len[r] < 0 || a.seq_len[r] > cap) atomicAdd(a.pool.skipped, 1ull);
        if (per > PER && (int32_t)blockIdx.x < split.ctas) find(a, divide(split.begin(blockIdx.x), segs));
    }

    // All threads: the request that holds tile y of the requests' line.
    __device__ __forceinline__ void find(const AttendArgs &a, int64_t y) {
        __shared__ int32_t s_r;
        __shared__ int64_t s_before;
        int64_t base = 0, total;
        for (int32_t c = 0; c < a.n_reqs && base <= y; c += 32 * WARPS) {
            const int32_t r = c + threadIdx.x;
            const int64_t mine = r < a.n_reqs ? Span<TOK>(a, r).tiles + EXTRA : 0, ex = base + cta_exclusive<WARPS>(mine, &total);
            if (ex <= y && y < ex + mine) {
                s_r = r;
                s_before = ex;
            }
            base += total;
        }
        __syncthreads();
        r0 = s_r;
        before0 = s_before;
    }

    // Whole warp: the first tile at or after place x of the line, to which x is moved.
    __device__ __forceinline__ Place<TOK, EXTRA> locate(const AttendArgs &a, int32_t segs, int64_t &x) const {
        const int lane = threadIdx.x & 31;
        const int64_t y = divide(x, segs);
        Place<TOK, EXTRA> p;
        if (per <= PER) {
            const int at = __ffs(__ballot_sync(~0u, upto > y)) - 1;
            int64_t left = upto;
            int32_t r = lane * per + per;
#pragma unroll
            for (int k = PER - 1; k >= 0; --k)
                if (k < per && left > y) left -= tiles[k], --r;    // back to the request that holds y
            p.r = __shfl_sync(~0u, r, at);
            p.before = __shfl_sync(~0u, left, at);
        } else {
            int32_t r = r0;
            int64_t before = before0;
            for (;;) {
                const int64_t n = r + lane < a.n_reqs ? Span<TOK>(a, r + lane).tiles + EXTRA : 0;
                const int64_t in = before + warp_inclusive(n);
                const uint32_t past = __ballot_sync(~0u, in > y);
                const int at = past ? __ffs(past) - 1 : 31;
                const int64_t to = __shfl_sync(~0u, in, at), here = __shfl_sync(~0u, n, at);
                if (past) {
                    p.r = r + at;
                    p.before = to - here;
                    break;
                }
                before = to;
                r += 32;
            }
        }
        p.request(a);
        const int64_t rest = x - p.before * segs;
        p.seg = (int32_t)divide(rest, p.tiles + EXTRA);
        p.tile = (int32_t)(rest - (int64_t)p.seg * (p.tiles + EXTRA));
        if (p.tile >= p.tiles) {
            x -= p.tile - (p.tiles - 1);
            p.tile = p.tiles - 1;
            p.next(a, segs, x);
        }
        return p;
    }
};

}  // namespace kvx
