// kvx_slot_map: block tables and slot maps from request lengths, in one launch.
//
// With had(r) = ceil(ctx / bs) and need(r) = ceil((ctx + new) / bs), request r takes the entries
// [B(r), B(r) + need - had) of the free list and its new tokens are [T(r), T(r) + new), B and T the
// exclusive sums of need - had and new over the requests before it.
//
// Every CTA takes the sums over all requests itself, kReqs at a time in shared memory, and then writes
// its share of the outputs: output tiles go round-robin over the CTAs, and a token or block finds its
// request by bisection of the sums. So nothing is handed from CTA to CTA and no scratch is needed; the
// repeated reads are 8 bytes per request and CTA, from L2.
#include "kvx_launch.cuh"

#include <algorithm>

namespace kvx {

constexpr int kSlotThreads = 256;
constexpr int kReqs = 1024;            // requests per pass over shared memory
constexpr int kTokTile = 2 * kSlotThreads;

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

__device__ __forceinline__ uint32_t blocks_of(uint32_t tokens, uint32_t bs) { return tokens ? (tokens - 1) / bs + 1 : 0; }

// First tile at or after `lo` that is this CTA's.
__device__ __forceinline__ int64_t first_tile(int64_t lo) {
    const int64_t g = gridDim.x;
    return lo + ((int64_t)blockIdx.x - lo % g + g) % g;
}

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
        Sums mine = {0, 0};
        for (int i = i0; i < i1; ++i) {
            const int32_t c = a.ctx_len[r0 + i], w = a.new_len[r0 + i];
            const int64_t ctx = max(c, 0), end = min(ctx + max(w, 0), inf);
            const uint32_t had = blocks_of((uint32_t)ctx, bs), need = blocks_of((uint32_t)end, bs);
            const uint32_t top = (uint32_t)a.max_blocks;
            bad |= c < 0 || w < 0 || ctx + w > inf || need > top;
            s_ctx[i] = (int32_t)ctx;
            s_had[i] = (int32_t)min(had, top);
            s_tok[i] = end - ctx;                        // turned into sums below
            s_blk[i] = min(need, top) - min(had, top);
            mine = mine + Sums{s_tok[i], s_blk[i]};
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
        for (int64_t tile = first_tile(base.blk / kSlotThreads); tile * kSlotThreads < b_end; tile += gridDim.x) {
            const int64_t b = tile * kSlotThreads + threadIdx.x;
            if (b < base.blk || b >= b_end) continue;
            const int i = last_at_most(s_blk, m, b - base.blk);
            const int64_t col = s_had[i] + (b - base.blk - s_blk[i]);
            a.block_table[(r0 + i) * a.table_stride + col] = b < a.n_free ? a.free_blocks[b] : -1;
        }

        const int64_t t_end = min(base.tok + total.tok, a.max_tokens);
        for (int64_t tile = first_tile(base.tok / kTokTile); tile * kTokTile < t_end; tile += gridDim.x) {
            const int64_t t0 = tile * kTokTile + 2 * threadIdx.x;
            int64_t slot[2] = {-1, -1};
            int32_t pos[2] = {0, 0};
            if (t0 + 1 < base.tok || t0 >= t_end) continue;
            int i = last_at_most(s_tok, m, max(t0, base.tok) - base.tok);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t t = t0 + u - base.tok;
                if (t < 0 || t0 + u >= t_end) continue;
                while (i + 1 < m && s_tok[i + 1] <= t) ++i;
                pos[u] = s_ctx[i] + (int32_t)(t - s_tok[i]);
                const int32_t col = (int32_t)((uint32_t)pos[u] / bs), had = s_had[i];
                int32_t blk = -1;
                if (col < had) blk = a.block_table[(r0 + i) * a.table_stride + col];
                else if (col < a.max_blocks) {
                    const int64_t b = base.blk + s_blk[i] + (col - had);
                    if (b < a.n_free) blk = a.free_blocks[b];
                }
                if (blk >= 0) slot[u] = (int64_t)blk * bs + (uint32_t)(pos[u] - col * (int32_t)bs);
            }
            if (pairs && t0 >= base.tok && t0 + 1 < t_end) {
                *reinterpret_cast<longlong2 *>(a.slots + t0) = make_longlong2(slot[0], slot[1]);
                if (a.positions) *reinterpret_cast<int2 *>(a.positions + t0) = make_int2(pos[0], pos[1]);
            } else {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (t0 + u >= base.tok && t0 + u < t_end) {
                        a.slots[t0 + u] = slot[u];
                        if (a.positions) a.positions[t0 + u] = pos[u];
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
    const int64_t tiles = std::max((a.max_tokens + kTokTile - 1) / kTokTile, (int64_t)(a.n_reqs + 1023) / 1024);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, 4 * sms));
    return launch_after(kvx_slot_map_kernel, dim3(grid), kSlotThreads, 0, stream, a);
}

}  // namespace kvx
