// The decode side on the host: the typed pool handle (kvx_cache_*), argument checks and launches of the
// slot map, the append and the attention. The kernels are in kvx_slots.cu, kvx_append.cu and
// kvx_attend.cu.
#include "kvx_internal.h"

#include <algorithm>
#include <cmath>
#include <limits>
#include <new>

using namespace kvx;

static bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

void kvx::divisor(uint32_t d, uint32_t *mul, uint32_t *shift) {
    uint32_t s = 0;
    while (((uint64_t)1 << s) < d) ++s;
    *shift = s;
    *mul = (uint32_t)(((((uint64_t)1 << s) - d) << 32) / d + 1);
}

// Multiprocessors of the current device, asked for once.
kvx_status kvx::device_sms(int32_t *device, int32_t *sms) {
    static std::atomic<int32_t> known[64];
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev < 64) n = known[dev].load(std::memory_order_relaxed);
    if (e == cudaSuccess && !n) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    *device = dev;
    *sms = n;
    return KVX_OK;
}

// Maps of the rows of latents for kvx_latent_tensor.cu, where it can take them: one shard, in device memory, and rows that
// end with a head or heads of exactly the elements that it reads, since what lies beyond has to read as zero.
static void encode_rows(kvx_cache_t c) {
    const Geom &g = c->g;
    const bool hnd = g.layout == KVX_LAYOUT_HND;
    const int64_t rows = g.n_blocks * g.block_size * (hnd ? g.heads_per_shard : 1);
    if (g.n_planes != 1 || g.n_shards != 1 || c->outside_device || rows < 1 ||
        rows >= std::numeric_limits<int32_t>::max() || (!hnd && g.heads_per_shard > 1 && g.head_dim != kCacheMaxLatent))
        return;
    const int64_t row_bytes = hnd ? g.head_bytes() : g.row_bytes();
    int32_t run = 128 / g.elem_bytes;
    while (g.block_size % run) run /= 2;
    std::vector<RowMaps> maps(c->base.size());
    for (size_t i = 0; i < maps.size(); ++i)
        if (!encode_rows_map(c->base[i], rows, row_bytes, 128, run, &maps[i].run128) ||
            !encode_rows_map(c->base[i], rows, row_bytes, 64, run, &maps[i].run64) ||
            !encode_rows_map(c->base[i], rows, row_bytes, 128, 1, &maps[i].row128) ||
            !encode_rows_map(c->base[i], rows, row_bytes, 64, 1, &maps[i].row64))
            return;
    c->map_run = run;
    c->row_maps.swap(maps);
}

// Scratch of the handle, at the first call that runs on the device.
kvx_status kvx::cache_ready(kvx_cache_t c, cudaStream_t stream) {
    if (c->dev) {
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
        return dev == c->device ? KVX_OK : fail(KVX_EINVAL, "the cache was first used on device %d, the current one is %d", c->device, dev);
    }
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(stream, &cap);
    if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
    if (cap != cudaStreamCaptureStatusNone)
        return fail(KVX_EINVAL, "the first call on a cache allocates: make it before the capture");
    int32_t device = 0, sms = 0;
    kvx_status st = device_sms(&device, &sms);
    if (st) return st;
    int pageable = -1;
    for (size_t i = 0; i < c->base.size() && c->g.buf_bytes() > 0; ++i) {          // a buffer is a pointer of its own: each of them
        cudaPointerAttributes at;
        e = cudaPointerGetAttributes(&at, c->base[i]);
        if (e != cudaSuccess) return cuda_fail(e, "cudaPointerGetAttributes(cache buffer)");
        c->outside_device |= at.type != cudaMemoryTypeDevice;
        if (at.type != cudaMemoryTypeUnregistered) continue;
        if (pageable < 0 && (e = cudaDeviceGetAttribute(&pageable, cudaDevAttrPageableMemoryAccess, device)) != cudaSuccess)
            return cuda_fail(e, "cudaDeviceGetAttribute(pageable memory access)");
        if (!pageable) return fail(KVX_EINVAL, "a cache buffer is pageable host memory this GPU cannot access");
    }
    try {
        encode_rows(c);
    } catch (const std::bad_alloc &) {
        return fail(KVX_ENOMEM, "host allocation failed");
    }
    void *dev = nullptr;
    const size_t bases = c->base.size() * sizeof(void *), bytes = (256 + attend_scratch_bytes(sms, c->g.n_planes == 1) + 15) / 16 * 16;
    st = pool_alloc(&dev, bytes + bases, stream);
    if (st) return st;
    e = cudaMemsetAsync(dev, 0, bytes, stream);
    if (e == cudaSuccess) e = cudaMemcpyAsync((uint8_t *)dev + bytes, c->base.data(), bases, cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) {
        pool_free(dev);
        return cuda_fail(e, "preparing the cache's scratch");
    }
    c->dev = (uint8_t *)dev;
    c->dev_bases = (uint8_t *const *)(c->dev + bytes);
    c->device = device;
    c->sms = sms;
    return KVX_OK;
}

void kvx::cache_fill_layer(kvx_cache_t c, int32_t layer, CacheLayer *out) {
    const Geom &g = c->g;
    for (int32_t s = 0; s < g.n_shards; ++s) {
        void *const *at = c->base.data() + (size_t)layer * g.n_planes * g.n_shards + s;
        // a pool without blocks may have no memory: the kernels then copy nothing from this address
        out->k[s] = g.buf_bytes() ? (uint8_t *)at[0] : c->dev;
        out->v[s] = g.buf_bytes() ? (uint8_t *)at[g.n_planes == 2 ? g.n_shards : 0] : c->dev;
    }
    out->block_pitch = g.block_size * g.row_bytes();
    out->token_pitch = (int32_t)g.token_pitch();
    out->head_pitch = (int32_t)(g.layout == KVX_LAYOUT_HND ? g.block_size * g.head_bytes() : g.head_bytes());
    out->n_blocks = (int32_t)g.n_blocks;
    out->block_size = g.block_size;
    out->heads_per_shard = g.heads_per_shard;
    out->n_shards = g.n_shards;
    out->skipped = (unsigned long long *)c->dev;
}

kvx_status kvx::cache_check_layer(kvx_cache_t c, int32_t layer) {
    if (!c) return fail(KVX_EINVAL, "cache is NULL");
    if (layer < 0 || layer >= c->g.n_layers) return fail(KVX_EINVAL, "layer %d of %d", layer, c->g.n_layers);
    return KVX_OK;
}

// The arguments of kvx_cache_attend.
kvx_status kvx::cache_check_attend(kvx_cache_t c, int32_t layer, const void *q, int64_t q_stride, const int32_t *block_table,
                    int64_t table_stride, int32_t max_blocks, const int32_t *seq_len, int32_t n_reqs, void *out, int64_t out_stride, float *lse) {
    kvx_status st = cache_check_layer(c, layer);
    if (st) return st;
    const Geom &g = c->g;
    const kvx_cache_config &f = c->cfg;
    if (f.v_dim > kCacheMaxLatentValue) return fail(KVX_EUNSUPPORTED, "attention over latents with v_dim %d", f.v_dim);
    if (n_reqs < 0 || n_reqs > (1 << 24)) return fail(KVX_EINVAL, "n_reqs %d not in [0, 2^24]", n_reqs);
    if (max_blocks < 0 || table_stride < max_blocks) return fail(KVX_EINVAL, "max_blocks must be >= 0, table_stride >= max_blocks");
    if (n_reqs && (!q || !out || !seq_len || (max_blocks && !block_table)))
        return fail(KVX_EINVAL, "q, out, seq_len or block_table is NULL");
    if (n_reqs > 1 && (q_stride < (int64_t)f.n_q_heads * g.head_dim || out_stride < (int64_t)f.n_q_heads * f.v_dim))
        return fail(KVX_EINVAL, "strides below a request's elements");
    if (q_stride > ((int64_t)1 << 40) || out_stride > ((int64_t)1 << 40)) return fail(KVX_EINVAL, "stride above 2^40");
    if (!aligned16(q) || !aligned16(out) || (n_reqs > 1 && (q_stride % 8 || out_stride % 8)))
        return fail(KVX_EINVAL, "q and out: pointers and strides must be multiples of 16 bytes");
    if (((uintptr_t)block_table & 3) || ((uintptr_t)seq_len & 3) || ((uintptr_t)lse & 3))
        return fail(KVX_EINVAL, "an array is not on a boundary of its elements");
    return KVX_OK;
}

void kvx::cache_fill_attend(kvx_cache_t c, int32_t layer, const void *q, int64_t q_stride, const int32_t *block_table,
                    int64_t table_stride, int32_t max_blocks, const int32_t *seq_len, int32_t n_reqs, void *out, int64_t out_stride, float *lse,
                    AttendArgs *args) {
    const Geom &g = c->g;
    const kvx_cache_config &f = c->cfg;
    AttendArgs &a = *args;
    a = AttendArgs{};
    cache_fill_layer(c, layer, &a.pool);
    a.q = (const uint8_t *)q;
    a.out = (uint8_t *)out;
    a.lse = lse;
    a.block_table = block_table;
    a.seq_len = seq_len;
    a.q_stride = q_stride * 2;
    a.out_stride = out_stride * 2;
    a.table_stride = table_stride;
    a.max_blocks = max_blocks;
    a.n_reqs = n_reqs;
    a.n_q_heads = f.n_q_heads;
    a.n_kv_heads = g.n_shards * g.heads_per_shard;
    a.head_dim = g.head_dim;
    a.v_dim = f.v_dim;
    a.window = f.window;
    a.scale = (float)((double)f.scale * (double)f.k_scale * 1.4426950408889634);
    a.v_scale = f.v_scale;
    divisor((uint32_t)g.block_size, &a.block_mul, &a.block_shift);
    a.block_pitch16 = (uint32_t)(a.pool.block_pitch / 16);
    a.token_pitch16 = (uint32_t)(a.pool.token_pitch / 16);
    a.latent = g.n_planes == 1;
    a.row_maps = c->row_maps.empty() ? nullptr : &c->row_maps[(size_t)layer];
    a.map_run = c->map_run;
    const bool hnd = g.layout == KVX_LAYOUT_HND;
    a.map_rows = (int32_t)std::min<int64_t>(g.n_blocks * g.block_size * (hnd ? g.heads_per_shard : 1), std::numeric_limits<int32_t>::max());
    a.map_block = (uint32_t)(g.block_size * (hnd ? g.heads_per_shard : 1));
    a.map_head = hnd ? (uint32_t)g.block_size : 0;
    a.map_col = hnd ? 0 : (uint32_t)g.head_bytes();
    a.scratch = c->dev + 256;
    a.device = c->device;
}

extern "C" {

kvx_status kvx_slot_map(const int32_t *ctx_len, const int32_t *new_len, int32_t n_reqs, int32_t block_size,
                        const int32_t *free_blocks, int64_t n_free, int32_t *block_table, int64_t table_stride,
                        int32_t max_blocks, int64_t max_tokens, int64_t *tok_off, int64_t *slots,
                        int32_t *positions, int32_t *seq_len, kvx_slot_result *result, cudaStream_t stream) {
    if (n_reqs < 0 || n_reqs > (1 << 24)) return fail(KVX_EINVAL, "n_reqs %d not in [0, 2^24]", n_reqs);
    if (block_size < 1) return fail(KVX_EINVAL, "block_size must be >= 1");
    if (n_free < 0 || max_blocks < 0 || table_stride < max_blocks || max_tokens < 0)
        return fail(KVX_EINVAL, "n_free, max_blocks and max_tokens must be >= 0, table_stride >= max_blocks");
    if (max_tokens > ((int64_t)1 << 40)) return fail(KVX_EINVAL, "max_tokens above 2^40");
    if (!tok_off || !result) return fail(KVX_EINVAL, "tok_off and result are required");
    if (n_reqs && (!ctx_len || !new_len || !seq_len)) return fail(KVX_EINVAL, "a length array is NULL");
    if (n_reqs && max_blocks && !block_table) return fail(KVX_EINVAL, "block_table is NULL");
    if (n_free && !free_blocks) return fail(KVX_EINVAL, "free_blocks is NULL");
    if (max_tokens && !slots) return fail(KVX_EINVAL, "slots is NULL");
    if (((uintptr_t)slots & 7) || ((uintptr_t)tok_off & 7) || ((uintptr_t)result & 7) || ((uintptr_t)positions & 3) ||
        ((uintptr_t)seq_len & 3) || ((uintptr_t)ctx_len & 3) || ((uintptr_t)new_len & 3) || ((uintptr_t)block_table & 3) ||
        ((uintptr_t)free_blocks & 3))
        return fail(KVX_EINVAL, "an array is not on a boundary of its elements");
    if (n_reqs && (seq_len == ctx_len || seq_len == new_len)) return fail(KVX_EINVAL, "seq_len is an input array");
    int32_t device = 0, sms = 0;
    kvx_status st = device_sms(&device, &sms);
    if (st) return st;
    SlotArgs a = {ctx_len, new_len, free_blocks, block_table, positions, seq_len, tok_off, slots, result,
                  n_free, table_stride, max_tokens, n_reqs, block_size, max_blocks, 0, 0};
    divisor((uint32_t)block_size, &a.block_mul, &a.block_shift);
    const cudaError_t e = launch_slot_map(a, sms, stream);
    return e == cudaSuccess ? KVX_OK : cuda_fail(e, "launching the slot map");
}

kvx_status kvx_cache_create(const kvx_pool *pool, const kvx_cache_config *cfg, kvx_cache_t *out) {
    if (!out) return fail(KVX_EINVAL, "out is NULL");
    *out = nullptr;
    if (!cfg) return fail(KVX_EINVAL, "cfg is NULL");
    Geom g{};
    std::vector<void *> base;
    try {
        kvx_status st = read_geom(pool, "cache", &g, &base);
        if (st) return st;
    } catch (const std::bad_alloc &) {
        return fail(KVX_ENOMEM, "host allocation failed");
    }
    kvx_cache_config f = *cfg;
    for (int32_t r : f.reserved)
        if (r) return fail(KVX_EINVAL, "reserved fields must be 0");
    if (f.value_type != KVX_BF16 && f.value_type != KVX_F16 && f.value_type != KVX_E4M3)
        return fail(KVX_EINVAL, "unknown value_type %d", f.value_type);
    const bool f8 = f.value_type == KVX_E4M3;
    if (g.elem_bytes != (f8 ? 1 : 2)) return fail(KVX_EINVAL, "value_type %d with elem_bytes %d", f.value_type, g.elem_bytes);
    if (!f.io_type) f.io_type = f8 ? KVX_BF16 : f.value_type;
    if (f8 ? (f.io_type != KVX_BF16 && f.io_type != KVX_F16) : f.io_type != f.value_type)
        return fail(KVX_EINVAL, "io_type %d with value_type %d", f.io_type, f.value_type);
    if (g.n_planes > 2) return fail(KVX_EUNSUPPORTED, "a typed pool has 1 or 2 planes");
    const bool latent = g.n_planes == 1;
    if (g.n_shards > kCacheMaxShards) return fail(KVX_EUNSUPPORTED, "more than %d shards", kCacheMaxShards);
    const int64_t kv_heads = (int64_t)g.n_shards * g.heads_per_shard;
    if (!f.n_q_heads && kv_heads <= std::numeric_limits<int32_t>::max()) f.n_q_heads = (int32_t)kv_heads;
    if (f.n_q_heads < 1 || f.n_q_heads % kv_heads)
        return fail(KVX_EINVAL, "n_q_heads %d is not a multiple of %lld KV heads", f.n_q_heads, (long long)kv_heads);
    if (f.n_q_heads > 65536) return fail(KVX_EUNSUPPORTED, "more than 65536 query heads");
    if (!f.v_dim) f.v_dim = g.head_dim;
    if (f.v_dim < 1 || f.v_dim > g.head_dim || (!latent && f.v_dim != g.head_dim))
        return fail(KVX_EINVAL, "v_dim %d with head_dim %d and %d planes", f.v_dim, g.head_dim, g.n_planes);
    if (g.head_dim > (latent ? kCacheMaxLatent : kCacheMaxDim))
        return fail(KVX_EUNSUPPORTED, "head_dim %d with %d planes", g.head_dim, g.n_planes);
    if (g.head_bytes() % 16 || (int64_t)f.v_dim * g.elem_bytes % 16)
        return fail(KVX_EUNSUPPORTED, "head rows of %lld bytes are not whole 16-byte vectors", (long long)g.head_bytes());
    if (g.block_size * g.row_bytes() > std::numeric_limits<int32_t>::max())
        return fail(KVX_EUNSUPPORTED, "blocks of 2^31 bytes or more");
    if (g.buf_bytes() >= (int64_t)1 << 36) return fail(KVX_EUNSUPPORTED, "buffers of 64 GiB or more");
    for (void *p : base)
        if (!aligned16(p)) return fail(KVX_EUNSUPPORTED, "a buffer is not on a 16-byte boundary");
    if (f.window < 0) return fail(KVX_EINVAL, "window must be >= 0");
    for (float x : {f.scale, f.k_scale, f.v_scale})
        if (!std::isfinite(x) || x < 0) return fail(KVX_EINVAL, "scales must be finite and not negative");
    if (!f8 && ((f.k_scale && f.k_scale != 1.0f) || (f.v_scale && f.v_scale != 1.0f)))
        return fail(KVX_EINVAL, "16-bit values have no scale");
    if (!f.scale) f.scale = (float)(1.0 / std::sqrt((double)g.head_dim));
    if (!f.k_scale) f.k_scale = 1.0f;
    if (latent && f.v_scale && f.v_scale != f.k_scale) return fail(KVX_EINVAL, "one plane has one scale");
    if (!f.v_scale) f.v_scale = latent ? f.k_scale : 1.0f;
    if (!std::isfinite(1.0f / f.k_scale) || !std::isfinite(1.0f / f.v_scale))
        return fail(KVX_EINVAL, "a scale has no finite inverse");
    if (!std::isnormal((float)((double)f.scale * f.k_scale * 1.4426950408889634)))
        return fail(KVX_EINVAL, "scale * k_scale is out of range");
    kvx_cache_s *c = new (std::nothrow) kvx_cache_s;
    if (!c) return fail(KVX_ENOMEM, "host allocation failed");
    c->g = g;
    c->base.swap(base);
    c->cfg = f;
    *out = c;
    return KVX_OK;
}

kvx_status kvx_cache_destroy(kvx_cache_t c) {
    if (!c) return KVX_OK;
    kvx_status st = KVX_OK;
    if (c->dev) {
        const DeviceScope on_device(c->device);
        const cudaError_t e = cudaDeviceSynchronize();   // the scratch may be in use on any stream
        if (e != cudaSuccess) st = cuda_fail(e, "cudaDeviceSynchronize(destroy)");
        pool_free(c->dev);
    }
    delete c;
    return st;
}

kvx_status kvx_cache_append(kvx_cache_t c, int32_t layer, const void *k, int64_t k_stride, const void *v,
                            int64_t v_stride, const int64_t *slots, int64_t n_tokens, cudaStream_t stream) {
    kvx_status st = cache_check_layer(c, layer);
    if (st) return st;
    const Geom &g = c->g;
    if (n_tokens < 0 || n_tokens > std::numeric_limits<int32_t>::max())
        return fail(KVX_EINVAL, "n_tokens %lld not in [0, 2^31)", (long long)n_tokens);
    const bool latent = g.n_planes == 1;
    if (latent && v) return fail(KVX_EINVAL, "a one-plane pool takes no v");
    if (n_tokens && (!k || (!latent && !v) || !slots)) return fail(KVX_EINVAL, "k, v or slots is NULL");
    const int64_t row = (int64_t)g.n_shards * g.heads_per_shard * g.head_dim;
    if (n_tokens > 1 && (k_stride < row || (!latent && v_stride < row)))
        return fail(KVX_EINVAL, "strides below a token's %lld elements", (long long)row);
    if (k_stride > ((int64_t)1 << 40) || (!latent && v_stride > ((int64_t)1 << 40))) return fail(KVX_EINVAL, "stride above 2^40");
    if (!aligned16(k) || !aligned16(v) || (n_tokens > 1 && (k_stride % 8 || (!latent && v_stride % 8))))
        return fail(KVX_EINVAL, "k and v: pointers and strides must be multiples of 16 bytes");
    if (((uintptr_t)slots & 7) != 0) return fail(KVX_EINVAL, "slots is not on an 8-byte boundary");
    if (n_tokens == 0) return KVX_OK;
    if ((st = cache_ready(c, stream))) return st;
    AppendArgs a;
    cache_fill_layer(c, layer, &a.pool);
    a.k = (const uint8_t *)k;
    a.v = (const uint8_t *)v;
    a.k_stride = k_stride * 2;
    a.v_stride = v_stride * 2;
    a.slots = slots;
    a.n_tokens = n_tokens;
    a.n_rows = g.n_blocks * g.block_size;
    a.head_dim = g.head_dim;
    a.planes = g.n_planes;
    a.k_inverse = 1.0f / c->cfg.k_scale;
    a.v_inverse = 1.0f / c->cfg.v_scale;
    const cudaError_t e = launch_append(a, c->cfg.value_type, c->cfg.io_type, c->sms, stream);
    return e == cudaSuccess ? KVX_OK : cuda_fail(e, "launching the append");
}

kvx_status kvx_cache_attend(kvx_cache_t c, int32_t layer, const void *q, int64_t q_stride,
                            const int32_t *block_table, int64_t table_stride, int32_t max_blocks,
                            const int32_t *seq_len, int32_t n_reqs, void *out, int64_t out_stride, float *lse,
                            cudaStream_t stream) {
    kvx_status st = cache_check_attend(c, layer, q, q_stride, block_table, table_stride, max_blocks, seq_len, n_reqs, out, out_stride, lse);
    if (st) return st;
    if (n_reqs == 0) return KVX_OK;
    if ((st = cache_ready(c, stream))) return st;
    if (c->g.n_planes == 1 && c->outside_device) return fail(KVX_EUNSUPPORTED, "attention over latents outside device memory");
    AttendArgs a;
    cache_fill_attend(c, layer, q, q_stride, block_table, table_stride, max_blocks, seq_len, n_reqs, out, out_stride, lse, &a);
    a.stall = c->stall;
    a.wait_ns = a.stall ? kCacheStallWaitNs : kCacheWaitNs;
    c->stall = 0;
    const cudaError_t e = launch_attend(a, c->cfg.value_type, c->cfg.io_type, c->sms, stream);
    return e == cudaSuccess ? KVX_OK : cuda_fail(e, "launching the attention");
}

kvx_status kvx_cache_inject_stall(kvx_cache_t c, int32_t part) {
    if (!c) return fail(KVX_EINVAL, "cache is NULL");
    if (part < kStallScores || part > kStallCopies) return fail(KVX_EINVAL, "part %d not in [1, 4]", part);
    if (c->g.n_planes != 1) return fail(KVX_EUNSUPPORTED, "the stall hook is for caches of latents");
    c->stall = part;
    return KVX_OK;
}

kvx_status kvx_cache_status(kvx_cache_t c, cudaStream_t stream) {
    if (!c) return fail(KVX_EINVAL, "cache is NULL");
    cudaError_t e = cudaStreamSynchronize(stream);
    unsigned long long n[2] = {0, 0};
    if (e == cudaSuccess && c->dev) {
        e = cudaMemcpyAsync(n, c->dev, sizeof n, cudaMemcpyDeviceToHost, stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
        if (e == cudaSuccess && (n[0] || n[1])) {
            e = cudaMemsetAsync(c->dev, 0, sizeof n, stream);
            if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
        }
    }
    if (e != cudaSuccess) return cuda_fail(e, "kvx_cache_status");
    if (n[1]) return fail(KVX_ETIMEDOUT, "a copy into shared memory did not arrive: the outputs since the last check are not valid");
    if (n[0]) return fail(KVX_ERANGE, "%llu slots, blocks or lengths out of bounds were skipped", n[0]);
    return KVX_OK;
}

}  // extern "C"
