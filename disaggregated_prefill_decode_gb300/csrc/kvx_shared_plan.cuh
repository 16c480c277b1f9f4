// The plan of a batch's shared prefixes: what each group shares, and the units that kvx_shared.cuh multiplies.
#pragma once

#include "kvx_attend.cuh"

namespace kvx {

constexpr int kSharedTile = 128, kSharedRows = 128;                // positions of a tile, rows of a slot
constexpr int kSharedSwitch = 3;                                   // what a change of units counts, in places of the line
// Prefixes of fewer positions are read by each request: a tile of the tensor pipe is 128.
constexpr int32_t kSharedLeast = 128;

// Two places a tile where both slots take each tile, one where they take turns.
__host__ __device__ inline int shared_weight(int32_t rows) { return rows > kSharedRows ? 2 : 1; }
__host__ __device__ inline int32_t shared_tiles(int32_t tokens) { return (int32_t)(((uint32_t)tokens + kSharedTile - 1) / kSharedTile); }

__device__ __forceinline__ int32_t request_length(const AttendArgs &a, int32_t r) {
    return (int32_t)min((int64_t)max(a.seq_len[r], 0), (int64_t)a.max_blocks * a.pool.block_size);
}

// Whole warp: the positions that requests [lo, hi) share. A group of two members or more shares the first P positions, P what it
// names but at most its shortest member's length. With a window every member's has to reach the start, else each reads its own.
template <class Length> __device__ __forceinline__ int32_t shared_tokens(const AttendArgs &a, int32_t lo, int32_t hi, int32_t prefix, Length length) {
    int32_t least = INT32_MAX, most = 0;
    for (int32_t r = lo + (threadIdx.x & 31); r < hi; r += 32) {
        const int32_t len = length(r);
        least = min(least, len);
        most = max(most, len);
    }
    least = __reduce_min_sync(~0u, least);
    most = __reduce_max_sync(~0u, most);
    const int32_t tokens = hi - lo < 2 ? 0 : min(prefix, least);
    return tokens < kSharedLeast || (a.window && most > a.window) ? 0 : tokens;
}

template <int THREADS> struct PlanRoom {
    int64_t place[THREADS], sums[2][THREADS / 32];
    int32_t unit[THREADS];
};

// All threads of a CTA: the units of groups [g0, g0 + n), n up to THREADS, of which the first tokens[i] positions are shared (0: none),
// and where their requests find them; behind the places and units of the groups before.
template <int THREADS> __device__ __forceinline__ void plan_units(const SharedArgs &s, int32_t g0, int32_t n, const int32_t *tokens, int64_t &places,
                                                                  int64_t &units, PlanRoom<THREADS> &room) {
    const AttendArgs &a = s.a;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t group = a.n_q_heads / a.n_kv_heads;
    int64_t my_units = 0, my_places = 0;
    if ((int32_t)threadIdx.x < n && tokens[threadIdx.x]) {
        const int64_t rows = (int64_t)(s.group_off[g0 + threadIdx.x + 1] - s.group_off[g0 + threadIdx.x]) * group;
        const int64_t pairs = (rows + 2 * kSharedRows - 1) / (2 * kSharedRows), tiles = shared_tiles(tokens[threadIdx.x]);
        my_units = pairs * a.n_kv_heads;
        my_places = a.n_kv_heads * (pairs * kSharedSwitch + (pairs - 1) * 2 * tiles + tiles * shared_weight((int32_t)(rows - (pairs - 1) * 2 * kSharedRows)));
    }
    int64_t u = warp_inclusive(my_units), p = warp_inclusive(my_places);
    if (lane == 31) room.sums[0][w] = u, room.sums[1][w] = p;
    __syncthreads();
    int64_t all_units = 0, all_places = 0;
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i == w) u += all_units, p += all_places;
        all_units += room.sums[0][i];
        all_places += room.sums[1][i];
    }
    room.unit[threadIdx.x] = (int32_t)(units + u - my_units);
    room.place[threadIdx.x] = places + p - my_places;
    units += all_units;
    places += all_places;
    __syncthreads();
    for (int32_t i = w; i < n; i += THREADS / 32) {
        if (!tokens[i]) continue;
        const int32_t lo = s.group_off[g0 + i], hi = s.group_off[g0 + i + 1];
        const int32_t rows = (hi - lo) * group, pairs = (rows + 2 * kSharedRows - 1) / (2 * kSharedRows);
        const int64_t tiles = shared_tiles(tokens[i]), pair_places = 2 * tiles + kSharedSwitch;
        const int64_t head_places = (pairs - 1) * pair_places + tiles * shared_weight(rows - (pairs - 1) * 2 * kSharedRows) + kSharedSwitch;
        for (int32_t j = lane; j < pairs * a.n_kv_heads; j += 32) {
            const int32_t kvh = j / pairs, pair = j - kvh * pairs;
            SharedUnit x;
            x.begin = room.place[i] + kvh * head_places + pair * pair_places;
            x.first = lo;
            x.rows = min(rows - pair * 2 * kSharedRows, 2 * kSharedRows);
            x.pair = pair;
            x.kvh = kvh;
            x.tokens = tokens[i];
            x.pairs = pairs;
            if (room.unit[i] + j < s.max_units) s.units[room.unit[i] + j] = x;
        }
        for (int32_t r = lo + lane; r < hi; r += 32) s.place_of[r] = make_int4(tokens[i], room.unit[i], (r - lo) * group, pairs);
    }
    __syncthreads();
}

__device__ __forceinline__ void plan_header(const SharedArgs &s, int64_t places, int64_t units) {
    if (threadIdx.x == 0) {
        s.header->places = places;
        s.header->units = (int32_t)min(units, (int64_t)s.max_units);
    }
}

// Small batches, in the kernel over the requests' own positions: each CTA finds for itself what the groups share (into rest_start()), and the
// last one makes the plan, which spares a launch. True: this CTA is done. `smem` is free again afterwards.
template <int THREADS> __device__ __forceinline__ bool plan_few(const SharedArgs &s, uint8_t *smem) {
    struct Room {
        int32_t len[kRestFew], tokens[kRestFew], prefix[kRestFew], off[kRestFew + 1];
        PlanRoom<THREADS> plan;
    };
    Room &room = *reinterpret_cast<Room *>(smem);
    int32_t *const start = rest_start();
    const AttendArgs &a = s.a;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool plans = blockIdx.x == gridDim.x - 1;
    bool bad = false;
    for (int32_t r = threadIdx.x; r < a.n_reqs; r += THREADS) {
        room.len[r] = request_length(a, r);
        start[r] = 0;
        if (plans) s.place_of[r] = make_int4(0, 0, 0, 0);
    }
    for (int32_t g = threadIdx.x; g < s.n_groups; g += THREADS) {
        const int32_t lo = s.group_off[g], hi = s.group_off[g + 1];
        bad |= lo < 0 || hi < lo || hi > a.n_reqs;
        room.off[g] = lo;
        room.off[g + 1] = hi;                                      // the next one's beginning, the same value
        room.prefix[g] = s.prefix_len[g];
        if (plans && room.prefix[g] < 0) atomicAdd(a.pool.skipped, 1ull);
    }
    bad = __syncthreads_or(bad);
    if (!bad)
        for (int32_t g = w; g < s.n_groups; g += THREADS / 32) {
            const int32_t lo = room.off[g], hi = room.off[g + 1];
            const int32_t tokens = shared_tokens(a, lo, hi, room.prefix[g], [&](int32_t r) { return room.len[r]; });
            if (lane == 0) room.tokens[g] = tokens;
            if (tokens)
                for (int32_t r = lo + lane; r < hi; r += 32) start[r] = tokens;
        }
    __syncthreads();
    if (!plans) return false;
    if (bad && threadIdx.x == 0) atomicAdd(a.pool.skipped, 1ull);
    int64_t places = 0, units = 0;
    for (int32_t g0 = 0; !bad && g0 < s.n_groups; g0 += THREADS) plan_units<THREADS>(s, g0, min(THREADS, s.n_groups - g0), room.tokens + g0, places, units, room.plan);
    plan_header(s, places, units);
    return true;
}

}  // namespace kvx
