// kvx_cache_attend_shared on the host: argument checks, the workspace, and when a batch takes kvx_cache_attend instead. The kernels
// are in kvx_shared.cu, kvx_shared.cuh and kvx_attend_planes.cuh.
#include "kvx_internal.h"

#include <algorithm>
#include <limits>

using namespace kvx;

// What sharing a prefix can save has to be worth its launches: below this many bytes that requests would read again, which they mostly
// find in L2, each reads its own. One bound for all that the host knows; where a batch breaks even depends on how many of its units' 256 rows are filled
// and how many units there are besides, so some batches above it lose up to a fifth (8 bits in many small groups, the last ones here). On GB300, 8 KV heads of 128 with 8 query heads each (us, shared / each its own): bf16, one group of 8 on 4096 positions
// (113 MiB read again) 26.6 / 26.5, on 8192 (226) 28.6 / 42.8; one of 64 on 512 (142) 34 / 31; 4 groups of 4 on 2048 (99) 27.9 / 27.3, on 4096 (195)
// 35 / 44; 16 groups of 4 on 512 (108) 35 / 31, on 1024 (204) 44 / 47. 8 bits: one group of 8 on 8192 (113) 29.1 / 29.4, on 16384 (225) 35 / 47; 4 groups
// of 16 on 1024 (128) 36 / 32, on 2048 (248) 36 / 50; 4 groups of 4 on 8192 (193) 48.8 / 47.4; 16 groups of 4 on 2048 (198) 60 / 50.
static constexpr int64_t kWorthBytes = 144 << 20;

// Rows are counted in 32 bits, rounded up to whole units of 256.
static bool can_share(const kvx_cache_t c, int32_t n_reqs) {
    return c->g.n_planes == 2 && c->g.head_dim <= kSharedMaxDim && (int64_t)n_reqs * c->cfg.n_q_heads <= std::numeric_limits<int32_t>::max() - 255;
}

// Places in the workspace; with `base` NULL only their size.
static int64_t lay_out(const kvx_cache_t c, int32_t n_reqs, int32_t n_groups, int32_t sms, uint8_t *base, SharedArgs *s) {
    const Geom &g = c->g;
    const int64_t kv_heads = (int64_t)g.n_shards * g.heads_per_shard, group = c->cfg.n_q_heads / kv_heads;
    const int64_t rows = (int64_t)n_reqs * c->cfg.n_q_heads;
    // a group has at most one unit of fewer than 256 rows for each KV head, and two members at least
    const int64_t units = kv_heads * (std::min(n_groups, n_reqs / 2) + n_reqs * group / 256);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t from = at;
        at += (bytes + 255) / 256 * 256;
        return base + from;
    };
    uint8_t *const header = take(sizeof(SharedHeader)), *const unit = take(units * (int64_t)sizeof(SharedUnit));
    uint8_t *const start = take(4 * (int64_t)n_reqs), *const place_of = take(16 * (int64_t)n_reqs);
    uint8_t *const ml = take(rows * 16), *const rest = take(rows * g.head_dim * 4), *const rest_parts = take(sms * rest_part_bytes(g.head_dim));
    uint8_t *const parts = take((units + sms) * shared_part_bytes(g.head_dim));
    if (s) {
        s->header = (SharedHeader *)header;
        s->units = (SharedUnit *)unit;
        s->max_units = (int32_t)std::min<int64_t>(units, std::numeric_limits<int32_t>::max());
        s->start = (int32_t *)start;
        s->place_of = (int4 *)place_of;
        s->parts = parts;
        s->a.start = s->start;
        s->a.rest = (float *)rest;
        s->a.rest_ml = (float4 *)ml;
        s->a.rest_parts = rest_parts;
    }
    return at;
}

extern "C" {

kvx_status kvx_cache_shared_bytes(kvx_cache_t c, int32_t n_reqs, int32_t n_groups, int64_t *bytes) {
    if (!c) return fail(KVX_EINVAL, "cache is NULL");
    if (!bytes) return fail(KVX_EINVAL, "bytes is NULL");
    if (n_reqs < 0 || n_reqs > (1 << 24) || n_groups < 0 || n_groups > (1 << 24)) return fail(KVX_EINVAL, "n_reqs or n_groups not in [0, 2^24]");
    *bytes = 0;
    if (n_reqs < 2 || n_groups < 1 || !can_share(c, n_reqs)) return KVX_OK;
    int32_t device = 0, sms = 0;
    const kvx_status st = device_sms(&device, &sms);
    if (st) return st;
    *bytes = lay_out(c, n_reqs, n_groups, sms, nullptr, nullptr);
    return KVX_OK;
}

kvx_status kvx_cache_attend_shared(kvx_cache_t c, int32_t layer, const void *q, int64_t q_stride, const int32_t *block_table,
                                   int64_t table_stride, int32_t max_blocks, const int32_t *seq_len, int32_t n_reqs,
                                   const int32_t *group_off, const int32_t *prefix_len, int32_t n_groups, void *out, int64_t out_stride,
                                   float *lse, void *workspace, int64_t workspace_bytes, cudaStream_t stream) {
    SharedArgs s{};
    kvx_status st = cache_check_attend(c, layer, q, q_stride, block_table, table_stride, max_blocks, seq_len, n_reqs, out, out_stride, lse);
    if (st) return st;
    if (n_groups < 0 || n_groups > (1 << 24)) return fail(KVX_EINVAL, "n_groups %d not in [0, 2^24]", n_groups);
    if (n_groups && (!group_off || !prefix_len)) return fail(KVX_EINVAL, "group_off or prefix_len is NULL");
    if (((uintptr_t)group_off & 3) || ((uintptr_t)prefix_len & 3)) return fail(KVX_EINVAL, "an array is not on a boundary of its elements");
    if (workspace_bytes < 0 || (uintptr_t)workspace & 15) return fail(KVX_EINVAL, "the workspace is not on a 16-byte boundary, or its size negative");
    if (n_reqs == 0) return KVX_OK;
    const Geom &g = c->g;
    const int64_t token = 2 * (int64_t)g.n_shards * g.row_bytes(), cap = (int64_t)max_blocks * g.block_size;
    const bool shares = n_reqs > 1 && n_groups && can_share(c, n_reqs);
    int64_t need = 0;
    if (shares) {
        if ((st = kvx_cache_shared_bytes(c, n_reqs, n_groups, &need))) return st;
        if (!workspace || workspace_bytes < need)
            return fail(KVX_EINVAL, "a workspace of %lld bytes is needed (kvx_cache_shared_bytes)", (long long)need);
    }
    const int64_t again = n_reqs - std::min(n_groups, n_reqs / 2);     // of each group's members all but one
    if (!shares || cap <= kWorthBytes / token / again)
        return kvx_cache_attend(c, layer, q, q_stride, block_table, table_stride, max_blocks, seq_len, n_reqs, out, out_stride, lse, stream);
    if ((st = cache_ready(c, stream))) return st;
    cache_fill_attend(c, layer, q, q_stride, block_table, table_stride, max_blocks, seq_len, n_reqs, out, out_stride, lse, &s.a);
    lay_out(c, n_reqs, n_groups, c->sms, (uint8_t *)workspace, &s);
    s.group_off = group_off;
    s.prefix_len = prefix_len;
    s.n_groups = n_groups;
    s.a.stall = c->shared_stall;
    s.a.wait_ns = s.a.stall ? kCacheStallWaitNs : kCacheWaitNs;
    c->shared_stall = 0;
    const cudaError_t e = launch_attend_shared(s, c->cfg.value_type, c->cfg.io_type, c->sms, stream);
    return e == cudaSuccess ? KVX_OK : cuda_fail(e, "launching the attention over shared prefixes");
}

kvx_status kvx_cache_inject_shared_stall(kvx_cache_t c, int32_t part) {
    if (!c) return fail(KVX_EINVAL, "cache is NULL");
    if (part < kStallSharedProducts || part > kStallSharedCopies) return fail(KVX_EINVAL, "part %d not in [1, 3]", part);
    if (c->g.n_planes != 2) return fail(KVX_EUNSUPPORTED, "the stall hook is for caches of two planes");
    c->shared_stall = part;
    return KVX_OK;
}

}  // extern "C"
