// kvx_pages_free, kvx_pages_fork, kvx_pages_compact: what a batch's block tables say about its pages, and kvx_cache_copy.
//
// The first three are one launch each. Their steps depend on one another (count, then place), so they run in one cluster of up
// to 16 CTAs, whose barrier takes the place of a second launch; sums go from CTA to CTA through distributed shared memory. The
// flags of the pool's blocks are read as bits: a warp takes up to 1024 neighbouring blocks, lane i the bits of 32 of them, so that
// ranks come from population counts and ids are read and written in whole lines. Bound by latency: 4 to 8 barriers and the
// reads between them.
//
// Measured on GB300: free, 40 requests 6.4 us (12.4 with barriers of a cluster, which one CTA has no need of), 1024 sessions on 87000
// pages 15.4 (20.3); fork with its copies, 16 rows of 16 layers 8.7 (12.9), 128 beams 12.3 (16.0); compact with its copies, 12 requests 16.6
// (39.7 when each entry's move was searched in memory, not in shared memory); 2.7 GB of latents 463 (509).
#include "kvx_launch.cuh"

#include <cooperative_groups.h>

#include <algorithm>

namespace kvx {

namespace cg = cooperative_groups;

constexpr int kPageThreads = 1024, kPageWarps = kPageThreads / 32;
constexpr int kPageCluster = 16;                   // CTAs at most
constexpr int kEntries = 4;                        // table entries of a lane at a time
constexpr int kMovesShared = 4096;                 // moves that the remapping has in shared memory

// Blocks that a request holds by its length; bad where the length is negative or beyond its row.
__device__ __forceinline__ int32_t held_blocks(const TableArgs &t, int32_t r, bool &bad) {
    const int64_t len = t.seq_len[r], cap = (int64_t)t.max_blocks * t.block_size;
    bad |= len < 0 || len > cap;
    const uint32_t x = (uint32_t)min(max(len, (int64_t)0), cap);       // a length is below 2^31
    return x ? (int32_t)(((__umulhi(x - 1, t.block_mul) + x - 1) >> t.block_shift) + 1) : 0;
}

// All entries of n rows of `width` columns, kEntries columns of a row for each lane: f(row, first column of the lane's, 32 apart).
template <class F> __device__ __forceinline__ void for_entries(int32_t n, int32_t width, int rank, int ranks, F f) {
    const int chunks = (int)(((uint32_t)width + 32 * kEntries - 1) / (32 * kEntries)), lane = threadIdx.x & 31;   // a width may be 2^31 - 1
    const int64_t items = (int64_t)n * chunks, warps = (int64_t)ranks * kPageWarps;
    for (int64_t i = (int64_t)rank * kPageWarps + (threadIdx.x >> 5); i < items; i += warps) {
        const int32_t r = items >> 32 ? (int32_t)(i / chunks) : (int32_t)((uint32_t)i / (uint32_t)chunks);
        f(r, (int32_t)(i - (int64_t)r * chunks) * (32 * kEntries) + lane);
    }
}

// The words of 32 blocks' flags over the warps of a launch: a warp takes `words` neighbouring ones at a time, as few as keep all warps busy.
struct Words {
    int words;
    int64_t first, step;               // blocks: of this warp's first word, of all warps in a pass
    __device__ __forceinline__ Words(int64_t n, int rank, int ranks) {
        const int64_t warps = (int64_t)ranks * kPageWarps, all = (n + 31) / 32;
        words = (int)min((all + warps - 1) / warps, (int64_t)32);
        first = ((int64_t)rank * kPageWarps + (threadIdx.x >> 5)) * words * 32;
        step = warps * words * 32;
    }
};

// Bits of a warp's words from block `first` on: lane i has those of word i. Set where some request holds the block.
__device__ __forceinline__ uint32_t held_bits(const int32_t *refs, int64_t first, int64_t n, int words) {
    const int lane = threadIdx.x & 31;
    uint32_t mine = 0;
    for (int i0 = 0; i0 < words; i0 += 8) {
        int32_t x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t b = first + (i0 + i) * 32 + lane;
            x[i] = i0 + i < words && b < n ? __ldcg(refs + b) : 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t bits = __ballot_sync(~0u, x[i] > 0);
            if (lane == i0 + i) mine = bits;
        }
    }
    return mine;
}
// Of the blocks from `first` on those below `end`.
__device__ __forceinline__ uint32_t bits_below(int64_t first, int64_t end) {
    return end <= first ? 0 : end - first >= 32 ? ~0u : (1u << (end - first)) - 1;
}

// Exclusive sum over the CTA's threads, and the total.
__device__ __forceinline__ int64_t page_exclusive(int64_t x, int64_t *total) {
    __shared__ int64_t sums[kPageWarps];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int64_t s = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(~0u, s, d);
        if (lane >= d) s += o;
    }
    __syncthreads();
    if (lane == 31) sums[w] = s;
    __syncthreads();
    int64_t y = sums[lane], z = y;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(~0u, z, d);
        if (lane >= d) z += o;
    }
    *total = __shfl_sync(~0u, z, 31);
    return __shfl_sync(~0u, z - y, w) + s - x;
}

// The CTAs of a launch. Between them a barrier costs a microsecond, most of it the fence that makes their writes visible; a CTA
// alone is spared it.
struct Ctas {
    cg::cluster_group cluster = cg::this_cluster();
    int rank = cluster.block_rank(), n = cluster.num_blocks();
    int turn = 0;                      // of the numbers that sum() passes on: one is still read while the next is written
    __device__ __forceinline__ void sync() {
        if (n == 1) __syncthreads();
        else cluster.sync();
    }
    // The CTAs' numbers before this one's, and all of them, by one barrier.
    __device__ __forceinline__ int64_t sum(int64_t x, int64_t *total) {
        __shared__ int64_t mine[2];
        if (n == 1) {
            __syncthreads();
            *total = x;
            return 0;
        }
        if (threadIdx.x == 0) mine[turn] = x;
        cluster.sync();
        int64_t before = 0, all = 0;
        for (int i = 0; i < n; ++i) {
            const int64_t y = *cluster.map_shared_rank(&mine[turn], i);
            if (i < rank) before += y;
            all += y;
        }
        turn ^= 1;
        *total = all;
        return before;
    }
    // No CTA may end while others read what it passed on.
    __device__ __forceinline__ void end() {
        if (n > 1) cluster.sync();
    }
};

// Ids of set bits, or what else f does with (rank, id): all ids of a line of 32 at a time.
template <class F> __device__ __forceinline__ void for_bits(uint32_t mine, int64_t first, int64_t rank, int words, F f) {
    const int lane = threadIdx.x & 31;
    if (!__any_sync(~0u, mine)) return;
#pragma unroll 4
    for (int i = 0; i < words; ++i) {
        const uint32_t bits = __shfl_sync(~0u, mine, i);
        const int64_t at = __shfl_sync(~0u, rank, i);
        if (bits >> lane & 1) f(at + __popc(bits & ((1u << lane) - 1)), (int32_t)(first + i * 32 + lane));
    }
}

__global__ void __launch_bounds__(kPageThreads, 1) kvx_pages_free_kernel(const PageArgs a) {
    Ctas ctas;
    const int rank = ctas.rank, ranks = ctas.n;
    wait_for_earlier();
    for (int64_t b = (int64_t)rank * kPageThreads + threadIdx.x; b < a.n_blocks; b += (int64_t)ranks * kPageThreads) a.refs[b] = 0;
    ctas.sync();
    bool bad = false;
    for_entries(a.t.n_reqs, a.t.max_blocks, rank, ranks, [&](int32_t r, int32_t col) {
        const int32_t held = held_blocks(a.t, r, bad);
        const int32_t *row = a.t.block_table + r * a.t.table_stride;
        int32_t b[kEntries];
#pragma unroll
        for (int k = 0; k < kEntries; ++k) b[k] = col + 32 * k < held ? row[col + 32 * k] : -2;
#pragma unroll
        for (int k = 0; k < kEntries; ++k) {
            if (b[k] >= 0 && b[k] < a.n_blocks) atomicAdd(a.refs + b[k], 1);
            else bad |= b[k] != -2 || col + 32 * k < held;
        }
    });
    if (a.t.max_blocks == 0)                       // no entries: the lengths are looked at all the same
        for (int32_t r = rank * kPageThreads + threadIdx.x; r < a.t.n_reqs; r += ranks * kPageThreads) held_blocks(a.t, r, bad);
    int64_t any, n_free = 0;
    ctas.sum(__syncthreads_or(bad), &any);                             // its barrier orders the counts too
    const Words own(a.n_blocks, rank, ranks);
    const int lane = threadIdx.x & 31;
    for (int64_t pass = 0; pass < a.n_blocks; pass += own.step) {
        const int64_t first = pass + own.first;
        const uint32_t held = held_bits(a.refs, first, a.n_blocks, own.words);
        const uint32_t mine = lane < own.words ? ~held & bits_below(first + lane * 32, a.n_blocks) : 0;
        int64_t total, all;
        const int64_t before = page_exclusive(__popc(mine), &total), base = n_free + ctas.sum(total, &all);
        for_bits(mine, first, base + before, own.words, [&](int64_t k, int32_t id) { a.free_blocks[k] = id; });
        n_free += all;
    }
    if (rank == 0 && threadIdx.x == 0) *a.result = {a.n_blocks - n_free, n_free, any ? KVX_ERANGE : KVX_OK};
    ctas.end();
}

__global__ void __launch_bounds__(kPageThreads, 1) kvx_pages_fork_kernel(const ForkArgs a) {
    Ctas ctas;
    const int rank = ctas.rank, ranks = ctas.n;
    wait_for_earlier();
    const int64_t step = (int64_t)ranks * kPageThreads, t0 = (int64_t)rank * kPageThreads + threadIdx.x;
    for (int64_t r = t0; r < a.t.n_reqs; r += step) a.first[r] = INT32_MAX;
    ctas.sync();
    for (int64_t i = t0; i < a.n_out; i += step) {
        const int32_t p = a.parent[i];
        if (p >= 0 && p < a.t.n_reqs) atomicMin(a.first + p, (int32_t)i);
    }
    ctas.sync();
    bool bad = false;
    int64_t copies = 0, held_all = 0;
    for (int64_t pass = 0; pass < a.n_out; pass += step) {
        // a row for each thread: whether it needs a page of its own, and which
        const int64_t i = pass + t0;
        int32_t p = -1, held = 0, len = 0, last = -1;
        if (i < a.n_out) {
            p = a.parent[i];
            if (p < -1 || p >= a.t.n_reqs) bad = true, p = -1;
            if (p >= 0) {
                held = held_blocks(a.t, p, bad);
                len = (int32_t)min(max((int64_t)a.t.seq_len[p], (int64_t)0), (int64_t)a.t.max_blocks * a.t.block_size);
            }
        }
        bool need = held && held * (int64_t)a.t.block_size != len && __ldcg(a.first + p) != (int32_t)i;
        if (need) {
            last = a.t.block_table[p * a.t.table_stride + held - 1];
            if (last < 0) need = false;                                // a page that the row lacks, reported below
        }
        // both sums in one: pages to copy above, blocks below (at most 2^14 rows a pass, of 2^31 blocks)
        int64_t total, all;
        const int64_t in_cta = page_exclusive((int64_t)need << 46 | held, &total), in_all = ctas.sum(total, &all);
        const int64_t k = copies + ((in_all + in_cta) >> 46);
        int32_t to = -1;
        if (i < a.n_out) a.new_len[i] = len;
        if (need) {
            if (k < a.n_free) bad |= (to = a.free_blocks[k]) < 0;
            a.src[k] = to < 0 ? -1 : last;
            a.dst[k] = to < 0 ? -1 : to;
        }
        copies += all >> 46;
        held_all += all & (((int64_t)1 << 46) - 1);
        const int64_t upto = min(step, a.n_out - pass);
        int32_t signs = 0;
        for_entries((int32_t)upto, a.t.max_blocks, rank, ranks, [&](int32_t r, int32_t col) {
            const int32_t from = a.parent[pass + r];
            bool ignored = false;
            const bool any = from >= 0 && from < a.t.n_reqs;
            const int32_t n = any ? held_blocks(a.t, from, ignored) : 0;
            const int32_t *row = a.t.block_table + (any ? from * a.t.table_stride : 0);
            int32_t *out = a.new_table + (pass + r) * a.new_stride;
            int32_t b[kEntries];
#pragma unroll
            for (int e = 0; e < kEntries; ++e) b[e] = col + 32 * e < n ? row[col + 32 * e] : 0;
#pragma unroll
            for (int e = 0; e < kEntries; ++e) {
                signs |= b[e];
                if (col + 32 * e < a.t.max_blocks) out[col + 32 * e] = col + 32 * e < n ? b[e] : -1;
            }
        });
        bad |= signs < 0;                                              // a page that a parent's row lacks
        ctas.sync();                                                   // the row's last entry is written again, after its copy
        if (need) a.new_table[i * a.new_stride + held - 1] = to;
    }
    for (int64_t k = copies + t0; k < a.n_out; k += step) a.src[k] = a.dst[k] = -1;
    int64_t any;
    ctas.sum(__syncthreads_or(bad), &any);
    if (rank == 0 && threadIdx.x == 0) *a.result = {held_all, copies, copies > a.n_free ? KVX_ENOMEM : any ? KVX_ERANGE : KVX_OK};
    ctas.end();
}

__global__ void __launch_bounds__(kPageThreads, 1) kvx_pages_compact_kernel(const CompactArgs a) {
    __shared__ int32_t s_moves[2][kMovesShared];
    Ctas ctas;
    const int rank = ctas.rank, ranks = ctas.n;
    wait_for_earlier();
    const Words own(a.n_blocks, rank, ranks);
    const int lane = threadIdx.x & 31;
    const int64_t lane_at = lane * 32;
    // Up to a pass, as pools of up to half a million blocks are, the bits are read once.
    const bool once = a.n_blocks <= own.step;
    uint32_t bits = once ? held_bits(a.refs, own.first, a.n_blocks, own.words) : 0;
    // blocks held below `end`
    auto count = [&](int64_t end) {
        int64_t mine = 0, total, all;
        if (once) mine = __popc(bits & bits_below(own.first + lane_at, end));
        else
            for (int64_t first = own.first; first < end; first += own.step)
                mine += __popc(held_bits(a.refs, first, a.n_blocks, own.words) & bits_below(first + lane_at, end));
        page_exclusive(mine, &total);
        ctas.sum(total, &all);
        return all;
    };
    // With L blocks held, those held behind the first L go to the free ones among them: the free block b there has rank
    // b - (held before b), the held block b behind has rank (held before b) - (held below L).
    const int64_t held = count(a.n_blocks), below = count(held), moves = held - below;
    const bool fits = moves <= a.max_moves;
    int64_t base = 0;
    for (int64_t pass = 0; fits && pass < a.n_blocks; pass += own.step) {
        const int64_t first = pass + own.first;
        if (!once) bits = held_bits(a.refs, first, a.n_blocks, own.words);
        int64_t total, all;
        const int64_t in_cta = page_exclusive(__popc(bits), &total), before = base + ctas.sum(total, &all) + in_cta;
        base += all;
        const uint32_t front = lane < own.words ? bits_below(first + lane_at, held) : 0;
        const uint32_t holes = ~bits & front, movers = bits & ~front;
        if (!__any_sync(~0u, holes | movers)) continue;                // of this warp; the loop's barriers are above
        for_bits(holes, first, first + lane_at - before, own.words, [&](int64_t k, int32_t id) { a.dst[k] = id; });
        // ranks count held blocks alone: those of this lane's line that stand in the front come before its movers
        for_bits(movers, first, before + __popc(bits & front) - below, own.words, [&](int64_t k, int32_t id) { a.src[k] = id; });
    }
    const int64_t n = fits ? moves : 0;
    for (int64_t k = n + (int64_t)rank * kPageThreads + threadIdx.x; k < a.max_moves; k += (int64_t)ranks * kPageThreads) a.src[k] = a.dst[k] = -1;
    ctas.sync();
    bool bad = false;
    // The new id of a block from L on: it stands among the moves, which are ascending.
    auto remap = [&](const auto &src, const auto &dst) {
        for_entries(a.t.n_reqs, a.t.max_blocks, rank, ranks, [&](int32_t r, int32_t col) {
            const int32_t mine = held_blocks(a.t, r, bad);
            const int32_t *row = a.t.block_table + r * a.t.table_stride;
            int32_t *out = a.new_table + r * a.new_stride;
            int32_t b[kEntries], at[kEntries];
            bool moves[kEntries];
#pragma unroll
            for (int e = 0; e < kEntries; ++e) b[e] = col + 32 * e < a.t.max_blocks ? row[col + 32 * e] : -1;
#pragma unroll
            for (int e = 0; e < kEntries; ++e) {
                const bool in = col + 32 * e < mine;
                bad |= in && (b[e] < 0 || b[e] >= a.n_blocks);
                moves[e] = in && fits && b[e] >= held && b[e] < a.n_blocks;
                at[e] = 0;
            }
            if (moves[0] || moves[1] || moves[2] || moves[3]) {
                for (int32_t half = n > 0 ? 1 << (31 - __clz((int)n)) : 0; half; half >>= 1)   // how many are below, from the highest bit down
#pragma unroll
                    for (int e = 0; e < kEntries; ++e)
                        if (at[e] + half <= n && src(at[e] + half - 1) < b[e]) at[e] += half;
#pragma unroll
                for (int e = 0; e < kEntries; ++e) {
                    const bool found = moves[e] && at[e] < n && src(at[e]) == b[e];
                    bad |= moves[e] && !found;                         // the counts are not those of this table
                    if (found) b[e] = dst(at[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < kEntries; ++e)
                if (col + 32 * e < a.t.max_blocks) out[col + 32 * e] = b[e];
        });
    };
    if (n <= kMovesShared) {
        for (int k = threadIdx.x; k < n; k += kPageThreads) s_moves[0][k] = __ldcg(a.src + k), s_moves[1][k] = __ldcg(a.dst + k);
        __syncthreads();
        remap([&](int64_t k) { return s_moves[0][k]; }, [&](int64_t k) { return s_moves[1][k]; });
    } else
        remap([&](int64_t k) { return __ldcg(a.src + k); }, [&](int64_t k) { return __ldcg(a.dst + k); });
    int64_t any;
    ctas.sum(__syncthreads_or(bad), &any);
    if (rank == 0 && threadIdx.x == 0) *a.result = {held, moves, !fits ? KVX_ENOMEM : any ? KVX_ERANGE : KVX_OK};
    ctas.end();
}

// ------------------------------------------------------------------------------------------------
// kvx_cache_copy: whole pages, read and written once. Each CTA gathers the pairs that name a page, kPairs at a time, and the
// grid's warps take pieces of 4 KiB of their pages in turn, eight 16-byte loads of a lane in flight, four CTAs an SM: 2.7 GB of
// pages in 450 us, 6.1 TB/s (0.90 of the copy rate).
// ------------------------------------------------------------------------------------------------

constexpr int kCopyThreads = 256, kPairs = 4096, kPiece = 8 * 32;      // kPiece: 16-byte vectors

__global__ void __launch_bounds__(kCopyThreads) kvx_cache_copy_kernel(const PageCopyArgs a) {
    __shared__ int2 s_pairs[kPairs];
    __shared__ int32_t s_n, s_behind;
    wait_for_earlier();
    const int lane = threadIdx.x & 31;
    const int64_t pieces = (a.vectors + kPiece - 1) / kPiece, warps = (int64_t)gridDim.x * (kCopyThreads / 32);
    int64_t turn = (int64_t)(threadIdx.x >> 5) * gridDim.x + blockIdx.x;           // this warp's next piece, counted over all batches
    int64_t done = 0;
    for (int64_t p0 = 0; p0 < a.n_pairs; p0 += kPairs) {
        __syncthreads();
        if (threadIdx.x == 0) s_n = s_behind = 0;
        __syncthreads();
        const int all = (int)min((int64_t)kPairs, a.n_pairs - p0);
        int n = 0, behind = 0;                                         // pairs of this thread, and the place behind its last one
        for (int p = threadIdx.x; p < all; p += kCopyThreads) {
            const int32_t x = a.src[p0 + p], y = a.dst[p0 + p];
            const bool in = x >= 0 && x < a.n_blocks && y >= 0 && y < a.n_blocks;
            s_pairs[p] = in ? make_int2(x, y) : make_int2(-1, -1);
            if (in) ++n, behind = p + 1;
            else if ((x != -1 || y != -1) && blockIdx.x == 0) atomicAdd(a.skipped, 1ull);
        }
        n = __reduce_add_sync(~0u, n);
        behind = __reduce_max_sync(~0u, behind);
        if (lane == 0 && n) {
            atomicAdd(&s_n, n);
            atomicMax(&s_behind, behind);
        }
        __syncthreads();
        if (s_n != s_behind) {                                         // not all in front: to the front, in order, so that every CTA counts the same pieces
            if (threadIdx.x < 32) {
                int m = 0;
                for (int i = 0; i < s_behind; i += 32) {
                    const int2 x = i + lane < s_behind ? s_pairs[i + lane] : make_int2(-1, -1);
                    const uint32_t in = __ballot_sync(~0u, x.x >= 0);
                    if (x.x >= 0) s_pairs[m + __popc(in & ((1u << lane) - 1))] = x;
                    m += __popc(in);
                    __syncwarp();
                }
            }
            __syncthreads();
        }
        const int64_t items = (int64_t)s_n * a.n_bufs * pieces;
        for (; turn < done + items; turn += warps) {
            const int64_t i = turn - done, page = i / pieces;
            const int32_t pair = (int32_t)(page / a.n_bufs), buf = (int32_t)(page - (int64_t)pair * a.n_bufs);
            uint4 *const base = reinterpret_cast<uint4 *>(a.bufs[buf]);
            const int64_t v0 = (i - page * pieces) * kPiece + lane;
            const uint4 *from = base + s_pairs[pair].x * a.vectors;
            uint4 *to = base + s_pairs[pair].y * a.vectors;
            uint4 x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (v0 + k * 32 < a.vectors) x[k] = __ldcs(from + v0 + k * 32);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (v0 + k * 32 < a.vectors) __stcs(to + v0 + k * 32, x[k]);
        }
        done += items;
    }
}

// ------------------------------------------------------------------------------------------------

// As launch_after, in one cluster. Few table entries and blocks take one CTA, whose barriers are the CTA's own, more of them 8 or 16. Measured with
// 1, 8, 16 CTAs (us): free, 15 thousand of them 7.9, 9.0, 11.8; 31 thousand 13, 9.3, 11.9; 124 thousand 44, 11.9, 12.8; 249 thousand 85, 17.1, 15.4;
// compact, 15 thousand 13.9, 14.2, 20.1; 31 thousand 25.8, 15.5, 21.1; 124 thousand 150, 27.3, 25.9. A fork looks at half as much of the same
// table: 33 thousand 7.5, 7.9, 10.9; 66 thousand 11.4, 8.9, 10.9; 131 thousand 19.9, 10.1, 11.8; 525 thousand 71, 18.4, 17.0.
template <class A> static cudaError_t launch_cluster(void (*kernel)(A), int64_t work, const A &args, cudaStream_t stream) {
    static std::atomic<uint64_t> asked;                                // of this kernel's arguments: one type each
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(asked.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        asked.fetch_or(bit, std::memory_order_relaxed);
    }
    const unsigned ctas = work <= 16 * kPageThreads ? 1 : work <= 128 * kPageThreads ? 8 : kPageCluster;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPageThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kernel, args);
    if (e == cudaSuccess) count_launch();
    return e;
}

static int64_t entries(const TableArgs &t) { return (int64_t)t.n_reqs * t.max_blocks; }

cudaError_t launch_pages_free(const PageArgs &a, cudaStream_t stream) {
    return launch_cluster(kvx_pages_free_kernel, entries(a.t) + a.n_blocks, a, stream);
}
cudaError_t launch_pages_fork(const ForkArgs &a, cudaStream_t stream) {
    return launch_cluster(kvx_pages_fork_kernel, ((int64_t)a.n_out * a.t.max_blocks + a.t.n_reqs) / 2, a, stream);
}
cudaError_t launch_pages_compact(const CompactArgs &a, cudaStream_t stream) {
    return launch_cluster(kvx_pages_compact_kernel, entries(a.t) + a.n_blocks, a, stream);
}

cudaError_t launch_cache_copy(const PageCopyArgs &a, int32_t sms, cudaStream_t stream) {
    const int64_t pieces = (a.vectors + kPiece - 1) / kPiece * a.n_bufs * a.n_pairs;
    const int64_t ctas = std::min<int64_t>((pieces + kCopyThreads / 32 - 1) / (kCopyThreads / 32), 4 * sms);
    return launch_after(kvx_cache_copy_kernel, dim3((unsigned)ctas), kCopyThreads, 0, stream, a);
}

}  // namespace kvx
