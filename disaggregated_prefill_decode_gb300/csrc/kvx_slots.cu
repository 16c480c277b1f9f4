// kvx_slot_map: block tables and slot maps from request lengths, in one launch.
//
// With had(r) = ceil(ctx / bs) and need(r) = ceil((ctx + new) / bs), request r takes the entries
// [B(r), B(r) + need - had) of the free list and its new tokens are [T(r), T(r) + new), B and T the
// exclusive sums of need - had and new over the requests before it.
//
// Every CTA takes the sums over all requests itself, kReqs at a time in shared memory, and then writes
// its share of the outputs: output tiles go round-robin over the warps, and a tile finds its request by
// bisection of the sums (by the warp, then a lane among the requests of its tile). So nothing is handed
// from CTA to CTA and no scratch is needed; the repeated reads are 8 bytes per request and CTA, from L2.
//
// Measured on GB300: 4.5 M tokens of 256 sessions (54 MB) 13.9 us (two tokens a thread with a bisection of
// their own 32.5, a bisection for 256 tokens 16.4, 32-bit arithmetic for tiles of one request 13.9); 777
// requests with 140 thousand tokens 7.5; 16 decoding requests 5.0, which is what the host needs for a call.
// Bound by the two latencies before the first store where it is small, by issue (2.7 a clock) where it is large.
#include "kvx_launch.cuh"

#include <algorithm>

namespace kvx {

constexpr int kSlotThreads = 256;
constexpr int kReqs = 1024;            // requests per pass over shared memory (at most: warp_last_at_most)
constexpr int kTokTile = 256;          // tokens of a warp: two neighbours per lane, four times
constexpr int kTokRounds = kTokTile / 64;

struct Sums { int64_t tok, blk; };

__device__ __forceinline__ Sums operator+(Sums a, Sums b) { return {a.tok + b.tok, a.blk + b.blk}; }

// Exclusive sum over the CTA's threads; *total receives the whole.
__device__ __forceinline__ Sums cta_exclusive(Sums x, Sums *total) {
    __shared__ Sums warp_sum[kSlotThreads / 32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    Sums s = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sums o = {__shfl_up_sync(~0u, s.tok, d), __shfl_up_sync(~0u, s.blk, d)};
        if (lane >= d) s = s + o;
    }
    if (lane == 31) warp_sum[w] = s;
    __syncthreads();
    Sums before = {0, 0}, all = {0, 0};
#pragma unroll
    for (int i = 0; i < kSlotThreads / 32; ++i) {
        if (i == w) before = all;
        all = all + warp_sum[i];
    }
    *total = all;
    return {before.tok + s.tok - x.tok, before.blk + s.blk - x.blk};
}

// Last i in [0, n) with off[i] <= x, off[0] <= x.
__device__ __forceinline__ int last_at_most(const int64_t *off, int n, int64_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// The same by a whole warp, n up to 1024. x below off[0] has no answer: the ballot would be empty and the search leave the array.
__device__ __forceinline__ int warp_last_at_most(const int64_t *off, int n, int64_t x) {
    const int lane = threadIdx.x & 31, step = (n + 31) / 32;
    const int lo = (31 - __clz(__ballot_sync(~0u, lane * step < n && off[min(lane * step, n - 1)] <= x))) * step;
    return lo + 31 - __clz(__ballot_sync(~0u, lane < step && lo + lane < n && off[min(lo + lane, n - 1)] <= x));
}

__device__ __forceinline__ uint32_t blocks_of(const SlotArgs &a, uint32_t tokens) {
    return tokens ? ((__umulhi(tokens - 1, a.block_mul) + tokens - 1) >> a.block_shift) + 1 : 0;
}

// First tile at or after `lo` that is number `mine` of `of`.
__device__ __forceinline__ int64_t first_tile(int64_t lo, int64_t mine, int64_t of) { return lo + (mine - lo % of + of) % of; }

__global__ void __launch_bounds__(kSlotThreads) kvx_slot_map_kernel(const SlotArgs a) {
    __shared__ int64_t s_tok[kReqs], s_blk[kReqs];      // sums before each request, within the pass
    __shared__ int32_t s_ctx[kReqs], s_had[kReqs];
    wait_for_earlier();
    const uint32_t bs = (uint32_t)a.block_size;
    const int64_t inf = INT32_MAX;
    Sums base = {0, 0};
    bool bad = false;                                    // CTA 0: this thread saw a request out of range
    const bool pairs = ((uintptr_t)a.slots & 15) == 0 && ((uintptr_t)a.positions & 7) == 0;
    for (int32_t r0 = 0; r0 < a.n_reqs; r0 += kReqs) {
        const int m = min(kReqs, a.n_reqs - r0);
        const int per = (m + kSlotThreads - 1) / kSlotThreads;
        const int i0 = min(m, (int)threadIdx.x * per), i1 = min(m, i0 + per);
        int32_t c[kReqs / kSlotThreads], w[kReqs / kSlotThreads];
#pragma unroll
        for (int k = 0; k < kReqs / kSlotThreads; ++k) {
            c[k] = i0 + k < i1 ? a.ctx_len[r0 + i0 + k] : 0;
            w[k] = i0 + k < i1 ? a.new_len[r0 + i0 + k] : 0;
        }
        Sums mine = {0, 0};
#pragma unroll
        for (int k = 0; k < kReqs / kSlotThreads; ++k) {
            if (i0 + k >= i1) break;
            const int64_t ctx = max(c[k], 0), end = min(ctx + max(w[k], 0), inf);
            const uint32_t had = blocks_of(a, (uint32_t)ctx), need = blocks_of(a, (uint32_t)end), top = (uint32_t)a.max_blocks;
            bad |= c[k] < 0 || w[k] < 0 || ctx + w[k] > inf || need > top;
            s_ctx[i0 + k] = (int32_t)ctx;
            s_had[i0 + k] = (int32_t)min(had, top);
            s_tok[i0 + k] = end - ctx;                   // turned into sums below
            s_blk[i0 + k] = min(need, top) - min(had, top);
            mine = mine + Sums{s_tok[i0 + k], s_blk[i0 + k]};
        }
        Sums total;
        Sums at = cta_exclusive(mine, &total);
        for (int i = i0; i < i1; ++i) {
            const Sums n = {s_tok[i], s_blk[i]};
            s_tok[i] = at.tok;
            s_blk[i] = at.blk;
            at = at + n;
        }
        __syncthreads();

        for (int i = threadIdx.x; i < m; i += kSlotThreads)
            if ((i >> 8) % (int)gridDim.x == (int)blockIdx.x) {
                const int64_t end = i + 1 < m ? s_tok[i + 1] : total.tok;
                a.tok_off[r0 + i] = base.tok + s_tok[i];
                a.seq_len[r0 + i] = (int32_t)(s_ctx[i] + end - s_tok[i]);
            }

        const int64_t b_end = base.blk + total.blk;
        for (int64_t tile = first_tile(base.blk / kSlotThreads, blockIdx.x, gridDim.x); tile * kSlotThreads < b_end; tile += gridDim.x) {
            const int64_t b = tile * kSlotThreads + threadIdx.x;
            if (b < base.blk || b >= b_end) continue;
            const int i = last_at_most(s_blk, m, b - base.blk);
            const int64_t col = s_had[i] + (b - base.blk - s_blk[i]);
            a.block_table[(r0 + i) * a.table_stride + col] = b < a.n_free ? a.free_blocks[b] : -1;
        }

        const int64_t t_end = min(base.tok + total.tok, a.max_tokens);
        const int lane = threadIdx.x & 31, warps = gridDim.x * (kSlotThreads / 32);
        for (int64_t tile = first_tile(base.tok / kTokTile, (int64_t)(threadIdx.x >> 5) * gridDim.x + blockIdx.x, warps);
             max(tile * kTokTile, base.tok) < t_end; tile += warps) {                 // a pass may add no token, or none below max_tokens
            const int64_t first = tile * kTokTile, from = max(first, base.tok), upto = min(first + kTokTile, t_end);
            const int r_lo = warp_last_at_most(s_tok, m, from - base.tok), r_hi = warp_last_at_most(s_tok, m, upto - 1 - base.tok);
            if (pairs && r_lo == r_hi && from == first && upto == first + kTokTile) {
                // all of one request, as nearly all tiles of a long prompt: 32 bits, and a third of the instructions
                const int32_t p0 = s_ctx[r_lo] + (int32_t)(from - base.tok - s_tok[r_lo]) + 2 * lane, had = s_had[r_lo];
                const int64_t b0 = base.blk + s_blk[r_lo];         // of the free list: the request's first new block
                const int32_t end = (int32_t)min((int64_t)a.max_blocks, had + max(a.n_free - b0, (int64_t)0));      // of the blocks it gets
                const int32_t *const old = a.block_table + (r0 + r_lo) * a.table_stride, *const fresh = a.free_blocks + (b0 - had);
                auto block = [&](int32_t col) { return col >= end ? -1 : col < had ? old[col] : fresh[col]; };
                int32_t blk[kTokRounds], next[kTokRounds], rest[kTokRounds];
#pragma unroll
                for (int u = 0; u < kTokRounds; ++u) {
                    const uint32_t p = (uint32_t)(p0 + 64 * u), col = (__umulhi(p, a.block_mul) + p) >> a.block_shift;
                    rest[u] = (int32_t)(p - col * bs);
                    blk[u] = block((int32_t)col);
                    next[u] = rest[u] + 1 == (int32_t)bs ? block((int32_t)col + 1) : blk[u];
                }
                longlong2 *const slots = reinterpret_cast<longlong2 *>(a.slots + first) + lane;
#pragma unroll
                for (int u = 0; u < kTokRounds; ++u)
                    slots[32 * u] = make_longlong2(blk[u] < 0 ? -1 : (int64_t)blk[u] * a.block_size + rest[u],
                                                   next[u] < 0 ? -1 : (int64_t)next[u] * a.block_size + (rest[u] + 1 == (int32_t)bs ? 0 : rest[u] + 1));
                if (a.positions) {
                    int2 *const positions = reinterpret_cast<int2 *>(a.positions + first) + lane;
#pragma unroll
                    for (int u = 0; u < kTokRounds; ++u) positions[32 * u] = make_int2(p0 + 64 * u, p0 + 64 * u + 1);
                }
                continue;
            }
            int32_t blk[kTokRounds][2], rest[kTokRounds][2], pos[kTokRounds][2];
#pragma unroll
            for (int u = 0; u < kTokRounds; ++u) {
                const int64_t x = first - base.tok + 64 * u + 2 * lane;     // of the first of two tokens
                int i = r_lo;
                if (r_lo < r_hi) {                                 // the tile has tokens of several requests
                    int hi = r_hi + 1;
                    while (hi - i > 1) {
                        const int mid = (i + hi) >> 1;
                        if (s_tok[mid] <= x) i = mid; else hi = mid;
                    }
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    while (k && i < r_hi && s_tok[i + 1] <= x + 1) ++i;
                    const int32_t p = s_ctx[i] + (int32_t)(x + k - s_tok[i]), had = s_had[i];
                    const int32_t col = (int32_t)((__umulhi((uint32_t)p, a.block_mul) + (uint32_t)p) >> a.block_shift);
                    pos[u][k] = p;
                    rest[u][k] = p - col * (int32_t)bs;
                    blk[u][k] = -1;
                    if (k && rest[u][1] && x + 1 > s_tok[i]) blk[u][1] = blk[u][0];     // in the block of the token before
                    else if (x + k + base.tok >= from && x + k + base.tok < upto) {
                        const int64_t b = base.blk + s_blk[i] + (col - had);
                        if (col < had) blk[u][k] = a.block_table[(r0 + i) * a.table_stride + col];
                        else if (col < a.max_blocks && b < a.n_free) blk[u][k] = a.free_blocks[b];
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kTokRounds; ++u) {
                const int64_t t = first + 64 * u + 2 * lane;
                int64_t slot[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) slot[k] = blk[u][k] < 0 ? -1 : (int64_t)blk[u][k] * bs + rest[u][k];
                if (pairs && t >= from && t + 1 < upto) {
                    *reinterpret_cast<longlong2 *>(a.slots + t) = make_longlong2(slot[0], slot[1]);
                    if (a.positions) *reinterpret_cast<int2 *>(a.positions + t) = make_int2(pos[u][0], pos[u][1]);
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (t + k >= from && t + k < upto) {
                            a.slots[t + k] = slot[k];
                            if (a.positions) a.positions[t + k] = pos[u][k];
                        }
                }
            }
        }

        if (blockIdx.x == 0)                             // tokens that go on in a block the table lacks
            for (int i = threadIdx.x; i < m; i += kSlotThreads) {
                const int64_t end = i + 1 < m ? s_tok[i + 1] : total.tok;
                if (end > s_tok[i] && s_ctx[i] % bs && s_ctx[i] / bs < a.max_blocks)
                    bad |= a.block_table[(r0 + i) * a.table_stride + s_ctx[i] / bs] < 0;
            }
        base = base + total;
        __syncthreads();
    }
    for (int64_t t = base.tok + (int64_t)blockIdx.x * kSlotThreads + threadIdx.x; t < a.max_tokens;
         t += (int64_t)gridDim.x * kSlotThreads)
        a.slots[t] = -1;
    if (blockIdx.x == 0) {
        const bool range = __syncthreads_or(bad) || base.tok > a.max_tokens;
        if (threadIdx.x == 0) {
            a.tok_off[a.n_reqs] = base.tok;
            a.result->n_tokens = base.tok;
            a.result->n_blocks = base.blk;
            a.result->status = base.blk > a.n_free ? KVX_ENOMEM : range ? KVX_ERANGE : KVX_OK;
        }
    }
}

cudaError_t launch_slot_map(const SlotArgs &a, int32_t sms, cudaStream_t stream) {
    // a CTA for every 8 tiles, or 4 tokens a thread where there are few
    const int64_t tiles = std::max((a.max_tokens + 1023) / 1024, (int64_t)(a.n_reqs + 1023) / 1024);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, 4 * sms));
    return launch_after(kvx_slot_map_kernel, dim3(grid), kSlotThreads, 0, stream, a);
}

}  // namespace kvx
