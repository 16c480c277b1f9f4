// kvx_cache_attend_shared: the launches, the plan of a large batch, and the join of what the other kernels leave.
//
// Three launches: the requests' own positions, with the plan made by one of their CTAs (11 us for 16 x 400 positions, 22 for 64 x 500), the prefixes,
// the join (5 us for 16 requests of 64 heads, 8 for 64). 16 samples of a prompt of 8192 30.8 us in all, 64 requests on 32768 102, 96 8-bit
// requests in 12 groups 49.5; with the own positions joined in their kernel, as kvx_cache_attend does, 1.4, 1.4 and 0 us more. With more than kRestFew
// requests or groups the plan is a launch of its own before the others (2 to 2.4 us more).
// Of launches that start before the one ahead has ended the wait is all that is left; letting them start earlier still (launch_dependents)
// took SM time from it: 40 us, 47. A plan in each CTA of the prefixes' kernel took as long as one of its own: its reads are as cold there.
#include "kvx_shared.cuh"

namespace kvx {

constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32, kPlanLens = 4096;

int64_t shared_part_bytes(int32_t head_dim) { return 2 * kSharedRows * ((int64_t)head_dim * 4 + 8); }

// One CTA, for batches of more than kRestFew requests or groups. Groups that are no ascending stretches of the requests are reported,
// and then nothing is shared: the results are the same.
__global__ void __launch_bounds__(kPlanThreads, 1) kvx_shared_plan(const __grid_constant__ SharedArgs s) {
    __shared__ int32_t s_tokens[kPlanThreads];
    __shared__ PlanRoom<kPlanThreads> s_room;
    __shared__ int32_t s_len[kPlanLens];               // the first requests' lengths, read with the groups and not after them
    wait_for_earlier();
    const AttendArgs &a = s.a;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bool bad = false;
    for (int32_t r = threadIdx.x; r < min(a.n_reqs, kPlanLens); r += kPlanThreads) s_len[r] = request_length(a, r);
    for (int32_t g = threadIdx.x; g < s.n_groups; g += kPlanThreads) {
        const int32_t lo = s.group_off[g], hi = s.group_off[g + 1];
        bad |= lo < 0 || hi < lo || hi > a.n_reqs;
        if (s.prefix_len[g] < 0) atomicAdd(a.pool.skipped, 1ull);
    }
    for (int32_t r = threadIdx.x; r < a.n_reqs; r += kPlanThreads) {
        s.start[r] = 0;
        s.place_of[r] = make_int4(0, 0, 0, 0);
    }
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) atomicAdd(a.pool.skipped, 1ull);
    int64_t places = 0, units = 0;
    for (int32_t g0 = 0; !bad && g0 < s.n_groups; g0 += kPlanThreads) {
        const int32_t n = min(kPlanThreads, s.n_groups - g0);
        for (int32_t i = w; i < n; i += kPlanWarps) {                  // a warp a group: what it shares
            const int32_t lo = s.group_off[g0 + i], hi = s.group_off[g0 + i + 1];
            const int32_t tokens = shared_tokens(a, lo, hi, s.prefix_len[g0 + i], [&](int32_t r) { return r < kPlanLens ? s_len[r] : request_length(a, r); });
            if (lane == 0) s_tokens[i] = tokens;
            if (tokens)
                for (int32_t r = lo + lane; r < hi; r += 32) s.start[r] = tokens;
        }
        __syncthreads();
        plan_units<kPlanThreads>(s, g0, n, s_tokens, places, units, s_room);
    }
    plan_header(s, places, units);
}

// The join: a thread has four elements of a row (request, query head), the sums of its own positions and those of the CTAs that its
// unit went to, ten at a time: half of the 19 or 20 that one unit for each of 8 KV heads leaves on 152 SMs, so that two rounds take them all (the
// whole call for 16 samples and for 64 requests on a document, which have such units: 8 36.7 and 105.3 us, 10 35.6 and 103.9, 12 36.4 and 104.8, 20 36.0 and
// 111). Units in fewer parts take one round, of which the places beyond are predicated. Reads and writes are whole sectors: 8 rows x 4 float4 a warp.
template <int IO, int D> __global__ void __launch_bounds__(256) kvx_shared_join(const __grid_constant__ SharedArgs s, int ctas) {
    constexpr int C4 = D / 4, ROWS = 256 / C4, AT_ONCE = 10;
    wait_for_earlier();
    const AttendArgs &a = s.a;
    const int c = threadIdx.x / 8 % C4;
    const int64_t row = (int64_t)blockIdx.x * ROWS + (threadIdx.x & 7) + threadIdx.x / (8 * C4) * 8;
    if (row >= (int64_t)a.n_reqs * a.n_q_heads || c * 4 >= a.head_dim) return;
    const int32_t r = (int32_t)(row / a.n_q_heads), head = (int32_t)(row - (int64_t)r * a.n_q_heads), group = a.n_q_heads / a.n_kv_heads;
    const int32_t kvh = head / group, in_group = head - kvh * group;
    const int4 place = __ldcg(s.place_of + r);
    const int64_t places = s.header->places;
    const float4 mine = __ldcg(a.rest_ml + row);
    float4 o = __ldcg(reinterpret_cast<const float4 *>(a.rest + row * a.head_dim) + c);
    float top = mine.x, l = mine.y;
    if (l == 0.0f) {                                                   // no position of its own has a weight
        top = -INFINITY;
        o = make_float4(0, 0, 0, 0);
    }
    auto add = [&](const float2 *ml_at, const float4 *o_at, int64_t bytes, int32_t n) {
        for (int32_t x0 = 0; x0 < n; x0 += AT_ONCE) {
            float2 ml[AT_ONCE];
            float4 y[AT_ONCE];
            float up = top;
#pragma unroll
            for (int x = 0; x < AT_ONCE; ++x) {
                ml[x] = make_float2(-INFINITY, 0.0f);
                if (x0 + x < n) {
                    ml[x] = __ldcg(reinterpret_cast<const float2 *>(reinterpret_cast<const uint8_t *>(ml_at) + (x0 + x) * bytes));
                    y[x] = __ldcg(reinterpret_cast<const float4 *>(reinterpret_cast<const uint8_t *>(o_at) + (x0 + x) * bytes));
                }
            }
#pragma unroll
            for (int x = 0; x < AT_ONCE; ++x)
                if (ml[x].y != 0.0f) up = fmaxf(up, ml[x].x);
            const float ref = up == -INFINITY ? 0.0f : up, old = fast_exp2(top - ref);
            top = up;
            l *= old;
            o = make_float4(o.x * old, o.y * old, o.z * old, o.w * old);
#pragma unroll
            for (int x = 0; x < AT_ONCE; ++x)
                if (ml[x].y != 0.0f) {                                 // sums without weights were not written
                    const float by = fast_exp2(ml[x].x - ref);
                    l = fmaf(by, ml[x].y, l);
                    o = make_float4(fmaf(by, y[x].x, o.x), fmaf(by, y[x].y, o.y), fmaf(by, y[x].z, o.z), fmaf(by, y[x].w, o.w));
                }
        }
    };
    const float2 *ml_at = nullptr;
    const float4 *o_at = nullptr;
    int64_t bytes = 0;
    int32_t n = 0;
    if (place.x) {                                                     // a member of a group that shares
        const int32_t at = place.z + in_group, unit = place.y + kvh * place.w + at / (2 * kSharedRows);
        const SharedUnit u = s.units[unit];
        const int weight = shared_weight(u.rows);
        const Split split = shared_split(places, ctas);
        const int32_t from = split.cta_of(u.begin), upto = split.cta_of(u.begin + (int64_t)shared_tiles(u.tokens) * weight - 1);
        const int in_slot = at % kSharedRows, slot = weight == 2 ? at % (2 * kSharedRows) / kSharedRows : 0;
        bytes = part_bytes(a.head_dim);
        n = upto - from + 1;
        const uint8_t *const part = s.parts + (unit + from) * bytes + slot * (bytes / 2);
        ml_at = reinterpret_cast<const float2 *>(part) + in_slot;
        o_at = reinterpret_cast<const float4 *>(part + kSharedRows * 8) + c * kSharedRows + in_slot;
    }
    const int32_t more = __float_as_int(mine.w);
    for (int k = 0; k < 2; ++k) {                                      // the prefix, then what other CTAs have of the request's own positions
        add(ml_at, o_at, bytes, n);
        if (!more) break;
        bytes = rest_part_bytes(a.head_dim);
        n = more;
        const uint8_t *const part = a.rest_parts + __float_as_int(mine.z) * bytes;
        const int in_set = in_group % (group > 8 ? 16 : 8);
        ml_at = reinterpret_cast<const float2 *>(part) + in_set;
        o_at = reinterpret_cast<const float4 *>(part + kRestRows * 8 + (int64_t)in_set * a.head_dim * 4) + c;
    }
    const float inverse = l == 0.0f ? 0.0f : a.v_scale / l;
    *reinterpret_cast<uint2 *>(a.out + r * a.out_stride + ((int64_t)head * a.head_dim + c * 4) * 2) =
        l == 0.0f ? make_uint2(0, 0) : make_uint2(pack<IO>(o.x * inverse, o.y * inverse), pack<IO>(o.z * inverse, o.w * inverse));
    if (c == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
}

template <int IO> static cudaError_t launch_join(const SharedArgs &s, int32_t sms, cudaStream_t stream) {
    const int64_t rows = (int64_t)s.a.n_reqs * s.a.n_q_heads;
    if (s.a.head_dim <= 64) return launch_after(kvx_shared_join<IO, 64>, dim3((unsigned)((rows + 15) / 16)), 256, 0, stream, s, sms);
    return launch_after(kvx_shared_join<IO, 128>, dim3((unsigned)((rows + 7) / 8)), 256, 0, stream, s, sms);
}

static cudaError_t launch_prefixes(const SharedArgs &s, int32_t vt, bool bf16, int32_t sms, cudaStream_t stream) {
    if (vt == KVX_BF16) return launch_shared_bf16(s, sms, stream);
    if (vt == KVX_F16) return launch_shared_f16(s, sms, stream);
    return bf16 ? launch_shared_e4m3_bf16(s, sms, stream) : launch_shared_e4m3_f16(s, sms, stream);
}
static cudaError_t launch_rest(const SharedArgs &s, int32_t vt, bool bf16, int32_t sms, cudaStream_t stream) {
    if (vt == KVX_BF16) return launch_rest_bf16(s, sms, stream);
    if (vt == KVX_F16) return launch_rest_f16(s, sms, stream);
    return bf16 ? launch_rest_e4m3_bf16(s, sms, stream) : launch_rest_e4m3_f16(s, sms, stream);
}

cudaError_t launch_attend_shared(const SharedArgs &args, int32_t vt, int32_t io, int32_t sms, cudaStream_t stream) {
    SharedArgs s = args;
    const bool bf16 = io == KVX_BF16, few = s.a.n_reqs <= kRestFew && s.n_groups <= kRestFew;
    cudaError_t e;
    if (few) {                                                         // the plan is made beside the requests' own positions
        s.a.start = nullptr;
        e = launch_rest(s, vt, bf16, sms, stream);
        if (e == cudaSuccess) e = launch_prefixes(s, vt, bf16, sms, stream);
    } else {
        e = launch_after(kvx_shared_plan, dim3(1), kPlanThreads, 0, stream, s);
        if (e == cudaSuccess) e = launch_prefixes(s, vt, bf16, sms, stream);
        if (e == cudaSuccess) e = launch_rest(s, vt, bf16, sms, stream);
    }
    if (e != cudaSuccess) return e;
    return bf16 ? launch_join<KVX_BF16>(s, sms, stream) : launch_join<KVX_F16>(s, sms, stream);
}

}  // namespace kvx
