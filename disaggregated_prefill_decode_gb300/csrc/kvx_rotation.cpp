// Rotations of queries and keys on the host: the frequencies (kvx_rotation_*), argument checks and launch of
// kvx_cache_append_rotated. The kernel is in kvx_rotate.cu.
#include "kvx_internal.h"

#include <algorithm>
#include <cmath>
#include <limits>
#include <new>

using namespace kvx;

static constexpr double kPi = 3.14159265358979323846;

static bool positive(double x) { return std::isfinite(x) && x > 0; }
static bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// The frequency of pair i of `dim` / 2, in radians a position.
static double frequency(const kvx_rotation_config &f, int i) {
    const double plain = std::pow(f.base, -2.0 * i / f.dim);
    if (f.scaling == KVX_ROTATE_LINEAR) return plain / f.factor;
    if (f.scaling == KVX_ROTATE_BANDS) {
        // turns over the original context: below `low` it is stretched, above `high` kept
        const double t = std::min(1.0, std::max(0.0, (f.original * plain / (2 * kPi) - f.low) / (f.high - f.low)));
        return plain / f.factor * (1 - t) + plain * t;
    }
    if (f.scaling == KVX_ROTATE_YARN) {
        auto pair_of = [&](double turns) { return f.dim * std::log(f.original / (turns * 2 * kPi)) / (2 * std::log(f.base)); };
        const double lo = std::max(std::floor(pair_of(f.high)), 0.0), hi = std::min(std::ceil(pair_of(f.low)), f.dim - 1.0);
        const double t = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 1e-3)));
        return plain / f.factor * t + plain * (1 - t);
    }
    return plain;
}

extern "C" {

kvx_status kvx_rotation_create(const kvx_rotation_config *cfg, kvx_rotation_t *out) {
    if (!out) return fail(KVX_EINVAL, "out is NULL");
    *out = nullptr;
    if (!cfg) return fail(KVX_EINVAL, "cfg is NULL");
    kvx_rotation_config f = *cfg;
    for (int32_t r : f.reserved)
        if (r) return fail(KVX_EINVAL, "reserved fields must be 0");
    if (f.layout != KVX_ROTATE_HALVES && f.layout != KVX_ROTATE_PAIRS) return fail(KVX_EINVAL, "unknown layout %d", f.layout);
    if (f.scaling < KVX_ROTATE_PLAIN || f.scaling > KVX_ROTATE_YARN) return fail(KVX_EINVAL, "unknown scaling %d", f.scaling);
    if (f.begin < 0 || f.dim < 0 || f.norm_dim < 0) return fail(KVX_EINVAL, "begin, dim and norm_dim must be >= 0");
    if (f.begin % 8 || f.norm_dim % 8 || f.dim % (f.layout == KVX_ROTATE_PAIRS ? 8 : 16))
        return fail(KVX_EUNSUPPORTED, "begin and norm_dim must be multiples of 8, dim of 16 (8 for pairs)");
    if (std::max(f.begin, f.norm_dim) > kCacheMaxLatent) return fail(KVX_EUNSUPPORTED, "begin or norm_dim above %d", kCacheMaxLatent);
    if (f.dim > 2 * kRotateMaxPairs) return fail(KVX_EUNSUPPORTED, "more than %d elements turn", 2 * kRotateMaxPairs);
    if (f.base == 0) f.base = 10000;
    if (!std::isfinite(f.base) || f.base <= 1) return fail(KVX_EINVAL, "base must be above 1");
    if (f.scaling != KVX_ROTATE_PLAIN && (!std::isfinite(f.factor) || f.factor < 1)) return fail(KVX_EINVAL, "factor must be >= 1");
    if (f.scaling == KVX_ROTATE_YARN) {
        if (f.low == 0) f.low = 1;
        if (f.high == 0) f.high = 32;
    }
    if (f.scaling >= KVX_ROTATE_BANDS && (!positive(f.low) || !positive(f.high) || !positive(f.original) || f.high <= f.low))
        return fail(KVX_EINVAL, "low, high and original must be positive, low below high");
    if (!std::isfinite(f.magnitude) || f.magnitude < 0) return fail(KVX_EINVAL, "magnitude must be finite and not negative");
    if (f.magnitude == 0) f.magnitude = f.scaling == KVX_ROTATE_YARN ? 0.1 * std::log(f.factor) + 1 : 1;
    if (!std::isfinite(f.eps) || f.eps < 0) return fail(KVX_EINVAL, "eps must be finite and not negative");
    if (f.eps == 0) f.eps = 1e-6f;
    kvx_rotation_s *r = new (std::nothrow) kvx_rotation_s;
    if (!r) return fail(KVX_ENOMEM, "host allocation failed");
    r->cfg = f;
    for (int i = 0; i < f.dim / 2; ++i) {
        r->frequency[i] = frequency(f, i);
        const double turns = r->frequency[i] / (2 * kPi);
        r->turns[i] = (uint64_t)std::ldexp(turns - std::floor(turns), 64);
    }
    *out = r;
    return KVX_OK;
}

kvx_status kvx_rotation_destroy(kvx_rotation_t r) {
    delete r;
    return KVX_OK;
}

kvx_status kvx_rotation_get(kvx_rotation_t r, double *frequencies, int32_t cap, int32_t *n, double *magnitude) {
    if (!r) return fail(KVX_EINVAL, "rotation is NULL");
    if (cap < 0 || (cap && !frequencies)) return fail(KVX_EINVAL, "cap is negative, or frequencies NULL");
    for (int32_t i = 0; i < std::min(cap, r->cfg.dim / 2); ++i) frequencies[i] = r->frequency[i];
    if (n) *n = r->cfg.dim / 2;
    if (magnitude) *magnitude = r->cfg.magnitude;
    return KVX_OK;
}

kvx_status kvx_cache_append_rotated(kvx_cache_t c, int32_t layer, kvx_rotation_t rotation, const void *q, int64_t q_stride,
                                    const void *q_weight, void *q_out, int64_t q_out_stride, const void *k, int64_t k_stride,
                                    const void *k_weight, const void *v, int64_t v_stride, const int32_t *positions, const int64_t *slots,
                                    int64_t n_tokens, cudaStream_t stream) {
    kvx_status st = cache_check_layer(c, layer);
    if (st) return st;
    if (!rotation) return fail(KVX_EINVAL, "rotation is NULL");
    const Geom &g = c->g;
    const kvx_rotation_config &f = rotation->cfg;
    if (f.begin + f.dim > g.head_dim || f.norm_dim > g.head_dim)
        return fail(KVX_EINVAL, "the rotation is for heads of %d elements or more, not %d", std::max(f.begin + f.dim, f.norm_dim), g.head_dim);
    if (n_tokens < 0 || n_tokens > std::numeric_limits<int32_t>::max())
        return fail(KVX_EINVAL, "n_tokens %lld not in [0, 2^31)", (long long)n_tokens);
    const bool latent = g.n_planes == 1;
    if (latent && v) return fail(KVX_EINVAL, "a one-plane pool takes no v");
    if (n_tokens && (!k || (!latent && !v) || !slots || (f.dim && !positions))) return fail(KVX_EINVAL, "k, v, positions or slots is NULL");
    if (n_tokens && (q == nullptr) != (q_out == nullptr)) return fail(KVX_EINVAL, "q and q_out go together");
    const int64_t row = (int64_t)g.n_shards * g.heads_per_shard * g.head_dim, q_row = (int64_t)c->cfg.n_q_heads * g.head_dim;
    if (n_tokens > 1 && (k_stride < row || (!latent && v_stride < row) || (q && (q_stride < q_row || q_out_stride < q_row))))
        return fail(KVX_EINVAL, "strides below a token's elements");
    for (int64_t s : {k_stride, v_stride, q_stride, q_out_stride})
        if (s > ((int64_t)1 << 40)) return fail(KVX_EINVAL, "stride above 2^40");
    if (n_tokens > 1 && q && q == q_out && q_stride != q_out_stride) return fail(KVX_EINVAL, "q_out in the place of q has its stride");
    if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) || !aligned16(q_weight) || !aligned16(k_weight) ||
        (n_tokens > 1 && (k_stride % 8 || (!latent && v_stride % 8) || (q && (q_stride % 8 || q_out_stride % 8)))))
        return fail(KVX_EINVAL, "q, k, v, q_out and the weights: pointers and strides must be multiples of 16 bytes");
    if (((uintptr_t)slots & 7) || ((uintptr_t)positions & 3)) return fail(KVX_EINVAL, "an array is not on a boundary of its elements");
    if (n_tokens == 0) return KVX_OK;
    if ((st = cache_ready(c, stream))) return st;
    RotateArgs a;
    cache_fill_layer(c, layer, &a.pool);
    a.q = (const uint8_t *)q;
    a.k = (const uint8_t *)k;
    a.v = (const uint8_t *)v;
    a.q_weight = q ? (const uint8_t *)q_weight : nullptr;
    a.k_weight = (const uint8_t *)k_weight;
    a.q_out = (uint8_t *)q_out;
    a.q_stride = n_tokens > 1 ? q_stride * 2 : 0;
    a.k_stride = n_tokens > 1 ? k_stride * 2 : 0;
    a.v_stride = n_tokens > 1 ? v_stride * 2 : 0;
    a.out_stride = n_tokens > 1 ? q_out_stride * 2 : 0;
    a.positions = positions;
    a.slots = slots;
    a.n_tokens = n_tokens;
    a.n_rows = g.n_blocks * g.block_size;
    a.n_q_heads = q ? c->cfg.n_q_heads : 0;
    a.n_kv_heads = g.n_shards * g.heads_per_shard;
    a.head_dim = g.head_dim;
    a.planes = g.n_planes;
    a.begin = f.begin;
    a.turned = f.dim;
    a.device = c->device;
    a.pairs = f.layout == KVX_ROTATE_PAIRS;
    a.norm_dim = f.norm_dim ? f.norm_dim : g.head_dim;
    a.norm_inverse = 1.0f / a.norm_dim;
    a.eps = f.eps;
    a.magnitude = (float)f.magnitude;
    a.k_inverse = 1.0f / c->cfg.k_scale;
    a.v_inverse = 1.0f / c->cfg.v_scale;
    std::copy(rotation->turns, rotation->turns + kRotateMaxPairs, a.turns);
    const cudaError_t e = launch_rotate(a, c->cfg.value_type, c->cfg.io_type, c->sms, stream);
    return e == cudaSuccess ? KVX_OK : cuda_fail(e, "launching the rotation");
}

}  // extern "C"
