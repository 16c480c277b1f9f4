// Pages of a cache on the host: argument checks and launches of kvx_pages_free, kvx_pages_fork, kvx_pages_compact and
// kvx_cache_copy. The kernels are in kvx_pages.cu.
#include "kvx_internal.h"

#include <limits>

using namespace kvx;

static bool off_elements(std::initializer_list<const void *> arrays) {
    for (const void *p : arrays)
        if ((uintptr_t)p & 3) return true;
    return false;
}

// Whether two arrays of n rows of `width` entries share memory.
static bool share(const int32_t *p, int64_t p_stride, int64_t p_rows, const int32_t *q, int64_t q_stride, int64_t q_rows, int64_t width) {
    if (!p_rows || !q_rows || !width) return false;
    const int32_t *p_end = p + (p_rows - 1) * p_stride + width, *q_end = q + (q_rows - 1) * q_stride + width;
    return p < q_end && q < p_end;
}

static kvx_status read_table(const int32_t *block_table, int64_t table_stride, int32_t max_blocks, const int32_t *seq_len, int32_t n_reqs,
                             int32_t block_size, TableArgs *t) {
    if (n_reqs < 0 || n_reqs > (1 << 24)) return fail(KVX_EINVAL, "n_reqs %d not in [0, 2^24]", n_reqs);
    if (block_size < 1) return fail(KVX_EINVAL, "block_size must be >= 1");
    if (max_blocks < 0 || table_stride < max_blocks || table_stride > ((int64_t)1 << 36))
        return fail(KVX_EINVAL, "max_blocks must be >= 0, table_stride >= max_blocks and at most 2^36");
    if (n_reqs && (!seq_len || (max_blocks && !block_table))) return fail(KVX_EINVAL, "seq_len or block_table is NULL");
    if (off_elements({block_table, seq_len})) return fail(KVX_EINVAL, "an array is not on a boundary of its elements");
    *t = TableArgs{block_table, seq_len, table_stride, n_reqs, max_blocks, block_size, 0, 0};
    divisor((uint32_t)block_size, &t->block_mul, &t->block_shift);
    return KVX_OK;
}

extern "C" {

kvx_status kvx_pages_free(const int32_t *block_table, int64_t table_stride, int32_t max_blocks, const int32_t *seq_len, int32_t n_reqs,
                          int32_t block_size, int64_t n_blocks, int32_t *refs, int32_t *free_blocks, kvx_page_result *result,
                          cudaStream_t stream) {
    PageArgs a{};
    kvx_status st = read_table(block_table, table_stride, max_blocks, seq_len, n_reqs, block_size, &a.t);
    if (st) return st;
    if (n_blocks < 0 || n_blocks > std::numeric_limits<int32_t>::max()) return fail(KVX_EINVAL, "n_blocks %lld not in [0, 2^31)", (long long)n_blocks);
    if (!result || (n_blocks && (!refs || !free_blocks))) return fail(KVX_EINVAL, "refs, free_blocks or result is NULL");
    if (off_elements({refs, free_blocks}) || ((uintptr_t)result & 7)) return fail(KVX_EINVAL, "an array is not on a boundary of its elements");
    a.refs = refs;
    a.free_blocks = free_blocks;
    a.result = result;
    a.n_blocks = n_blocks;
    const cudaError_t e = launch_pages_free(a, stream);
    return e == cudaSuccess ? KVX_OK : cuda_fail(e, "launching the page count");
}

kvx_status kvx_pages_fork(const int32_t *block_table, int64_t table_stride, int32_t max_blocks, const int32_t *seq_len, int32_t n_reqs,
                          const int32_t *parent, int32_t n_out, int32_t block_size, const int32_t *free_blocks, int64_t n_free,
                          int32_t *new_table, int64_t new_stride, int32_t *new_len, int32_t *src_blocks, int32_t *dst_blocks,
                          int32_t *scratch, kvx_page_result *result, cudaStream_t stream) {
    ForkArgs a{};
    kvx_status st = read_table(block_table, table_stride, max_blocks, seq_len, n_reqs, block_size, &a.t);
    if (st) return st;
    if (n_out < 0 || n_out > (1 << 24)) return fail(KVX_EINVAL, "n_out %d not in [0, 2^24]", n_out);
    if (n_free < 0 || new_stride < max_blocks || new_stride > ((int64_t)1 << 36))
        return fail(KVX_EINVAL, "n_free must be >= 0, new_stride >= max_blocks and at most 2^36");
    if (!result || (n_reqs && !scratch) || (n_free && !free_blocks)) return fail(KVX_EINVAL, "result, scratch or free_blocks is NULL");
    if (n_out && (!parent || !new_len || !src_blocks || !dst_blocks || (max_blocks && !new_table)))
        return fail(KVX_EINVAL, "parent, new_table, new_len, src_blocks or dst_blocks is NULL");
    if (off_elements({parent, free_blocks, new_table, new_len, src_blocks, dst_blocks, scratch}) || ((uintptr_t)result & 7))
        return fail(KVX_EINVAL, "an array is not on a boundary of its elements");
    if (share(block_table, table_stride, n_reqs, new_table, new_stride, n_out, max_blocks) || share(seq_len, 1, n_reqs, new_len, 1, n_out, 1))
        return fail(KVX_EINVAL, "new_table and new_len may not overlap the rows they are made from");
    a.parent = parent;
    a.free_blocks = free_blocks;
    a.new_table = new_table;
    a.new_len = new_len;
    a.src = src_blocks;
    a.dst = dst_blocks;
    a.first = scratch;
    a.result = result;
    a.new_stride = new_stride;
    a.n_free = n_free;
    a.n_out = n_out;
    const cudaError_t e = launch_pages_fork(a, stream);
    return e == cudaSuccess ? KVX_OK : cuda_fail(e, "launching the fork");
}

kvx_status kvx_pages_compact(const int32_t *block_table, int64_t table_stride, int32_t max_blocks, const int32_t *seq_len, int32_t n_reqs,
                             int32_t block_size, const int32_t *refs, int64_t n_blocks, int32_t *new_table, int64_t new_stride,
                             int32_t *src_blocks, int32_t *dst_blocks, int64_t max_moves, kvx_page_result *result, cudaStream_t stream) {
    CompactArgs a{};
    kvx_status st = read_table(block_table, table_stride, max_blocks, seq_len, n_reqs, block_size, &a.t);
    if (st) return st;
    if (n_blocks < 0 || n_blocks > std::numeric_limits<int32_t>::max()) return fail(KVX_EINVAL, "n_blocks %lld not in [0, 2^31)", (long long)n_blocks);
    if (max_moves < 0 || max_moves > std::numeric_limits<int32_t>::max() || new_stride < max_blocks || new_stride > ((int64_t)1 << 36))
        return fail(KVX_EINVAL, "max_moves not in [0, 2^31), or new_stride not in [max_blocks, 2^36]");
    if (!result || (n_blocks && !refs) || (max_moves && (!src_blocks || !dst_blocks)) || (n_reqs && max_blocks && !new_table))
        return fail(KVX_EINVAL, "refs, new_table, src_blocks, dst_blocks or result is NULL");
    if (off_elements({refs, new_table, src_blocks, dst_blocks}) || ((uintptr_t)result & 7))
        return fail(KVX_EINVAL, "an array is not on a boundary of its elements");
    if ((new_table != block_table || new_stride != table_stride) && share(block_table, table_stride, n_reqs, new_table, new_stride, n_reqs, max_blocks))
        return fail(KVX_EINVAL, "new_table is the table itself or apart from it");
    a.refs = refs;
    a.new_table = new_table;
    a.src = src_blocks;
    a.dst = dst_blocks;
    a.result = result;
    a.new_stride = new_stride;
    a.n_blocks = n_blocks;
    a.max_moves = max_moves;
    const cudaError_t e = launch_pages_compact(a, stream);
    return e == cudaSuccess ? KVX_OK : cuda_fail(e, "launching the compaction");
}

kvx_status kvx_cache_copy(kvx_cache_t c, int32_t layer_begin, int32_t layer_end, const int32_t *src_blocks, const int32_t *dst_blocks,
                          int32_t n_pairs, cudaStream_t stream) {
    if (!c) return fail(KVX_EINVAL, "cache is NULL");
    const Geom &g = c->g;
    if (layer_begin < 0 || layer_end < layer_begin || layer_end > g.n_layers)
        return fail(KVX_EINVAL, "layers [%d, %d) of %d", layer_begin, layer_end, g.n_layers);
    if (n_pairs < 0) return fail(KVX_EINVAL, "n_pairs must be >= 0");
    if (n_pairs && (!src_blocks || !dst_blocks)) return fail(KVX_EINVAL, "src_blocks or dst_blocks is NULL");
    if (off_elements({src_blocks, dst_blocks})) return fail(KVX_EINVAL, "an array is not on a boundary of its elements");
    if (n_pairs == 0 || layer_end == layer_begin) return KVX_OK;
    const int64_t per_layer = (int64_t)g.n_planes * g.n_shards, n_bufs = per_layer * (layer_end - layer_begin);
    if (n_bufs > std::numeric_limits<int32_t>::max()) return fail(KVX_EUNSUPPORTED, "2^31 buffers or more");
    kvx_status st = cache_ready(c, stream);
    if (st) return st;
    PageCopyArgs a{};
    a.bufs = c->dev_bases + layer_begin * per_layer;
    a.src = src_blocks;
    a.dst = dst_blocks;
    a.n_blocks = g.n_blocks;
    a.vectors = g.block_size * g.row_bytes() / 16;
    a.n_bufs = (int32_t)n_bufs;
    a.n_pairs = n_pairs;
    a.skipped = (unsigned long long *)c->dev;
    const cudaError_t e = launch_cache_copy(a, c->sms, stream);
    return e == cudaSuccess ? KVX_OK : cuda_fail(e, "launching the page copy");
}

}  // extern "C"
