// spec_cache_attend.cu -- attention over the 8-bit key/value cache and the
// attention weight that each cached token received (spec_cache_attend,
// spec_cache_weigh).

#include "spec_cache.cuh"

using namespace specc;

namespace {

struct AttendArgs {
    spec_cache c;
    spec_cache_form f;
    const int32_t *lengths;
    const __nv_bfloat16 *q;
    int64_t q_stride[3];
    int n, heads;
    __nv_bfloat16 *out;
    float *lse;
    const float *lse_in;
    float *weights;
    uint32_t *status;
};

// Does query i (at index at) see token j < s.len?
__device__ __forceinline__ bool sees(const AttendArgs &a, const Seq &s, int b, int i, int j)
{
    const int at = s.len - s.m + i;
    bool see;
    if (!a.f.parent) {
        see = j <= at;
    } else {
        const int t = j - (s.len - s.m);
        int k = i;
        while (k > t && t >= 0) {
            const int p = k > 0 ? a.f.parent[(size_t)b * a.n + k] : -1;
            k = p < k ? p : -1;
        }
        see = t < 0 || k == t;
    }
    if (a.f.window > 0)
        see = see && j > at - a.f.window;
    return see || (a.f.prefix && j < a.f.prefix[b]);
}

// A row's query, scaled score of one token, for a lane that holds the token.
__device__ __forceinline__ float score(const AttendArgs &a, const float *q, int page, int h, int row, float slope,
                                       float pos_q, int j)
{
    const spec_cache &c = a.c;
    const uint8_t *k = (const uint8_t *)c.k + (size_t)page * c.k_stride[0] + (size_t)h * c.k_stride[1] +
                       (size_t)row * c.k_stride[2];
    float dot = 0.0f;
    for (int d = 0; d < c.dim; d += 2) {
        const float2 v = decode2(*(const uint16_t *)(k + d), c.code);
        dot += v.x * q[d] + v.y * q[d + 1];
    }
    float x = dot * (c.k_scale[(size_t)page * c.kv_heads + h] * a.f.scale);
    if (a.f.softcap > 0.0f)
        x = a.f.softcap * tanhf(x / a.f.softcap);
    if (a.f.slopes) {
        const float p = (float)(c.positions ? c.positions[((size_t)page * c.kv_heads + h) * c.block + row] : j);
        x -= slope * fabsf(pos_q - p);
    }
    return x;
}

__device__ __forceinline__ float query_position(const AttendArgs &a, int b, int h, int at)
{
    if (!a.c.positions)
        return (float)at;
    const int page = page_of(a.c, b, at / a.c.block);
    return page < 0 ? 0.0f : (float)a.c.positions[((size_t)page * a.c.kv_heads + h) * a.c.block + at % a.c.block];
}

// One warp per query row: a lane scores one token of every 32, then all lanes
// add the 32 tokens' values, each its own dimensions.
__global__ void __launch_bounds__(128) attend_kernel(const AttendArgs a)
{
    __shared__ float sq[4][128];
    const spec_cache &c = a.c;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, D = c.dim;
    const long long r = (long long)blockIdx.x * 4 + wid;
    if (r >= (long long)c.batch * a.n * a.heads)
        return;
    const int H = (int)(r % a.heads), i = (int)(r / a.heads % a.n), b = (int)(r / a.heads / a.n);
    const int h = H / (a.heads / c.kv_heads);
    const Seq s = sequence(c, a.lengths, a.f.num_new, a.n, b, true);
    if (!s.ok && lane == 0)
        report(a.status, SPEC_STATUS_BAD_LENGTH);
    if (a.f.parent && lane == 0 && i > 0 && i < s.m && (unsigned)a.f.parent[(size_t)b * a.n + i] >= (unsigned)i)
        report(a.status, SPEC_STATUS_BAD_TREE);
    float *q = sq[wid];
    for (int d = lane; d < D; d += 32)
        q[d] = __bfloat162float(a.q[b * a.q_stride[0] + i * a.q_stride[1] + H * a.q_stride[2] + d]);
    __syncwarp();
    const bool live = i < s.m;
    const float slope = a.f.slopes ? a.f.slopes[H] : 0.0f;
    const float pos_q = live && a.f.slopes ? query_position(a, b, h, s.len - s.m + i) : 0.0f;
    float m = -INFINITY, l = 0.0f, o[4] = {0, 0, 0, 0};
    for (int j0 = 0; live && j0 < s.len; j0 += 32) {
        const int j = j0 + lane;
        int page = -1;
        float x = -INFINITY;
        bool see = false;
        if (j < s.len) {
            page = page_of(c, b, j / c.block);
            see = sees(a, s, b, i, j);
            if (page < 0 && see)
                report(a.status, SPEC_STATUS_BAD_PAGE);
            see = see && page >= 0;
            if (see)
                x = score(a, q, page, h, j % c.block, slope, pos_q, j);
        }
        const bool nan = __any_sync(0xffffffffu, x != x);
        float top = nan ? NAN : x;
        for (int w = 16; w > 0; w >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        if (nan)
            top = NAN;
        if (top == -INFINITY)
            continue;
        const float now = nan ? NAN : fmaxf(m, top);
        const float keep = m == -INFINITY ? 0.0f : expf(m - now);
        const float p = see ? expf(x - now) : 0.0f;
        float add = p;
        for (int w = 16; w > 0; w >>= 1)
            add += __shfl_xor_sync(0xffffffffu, add, w);
        l = l * keep + add;
        m = now;
        for (int d = 0; d < 4; ++d)
            o[d] *= keep;
        for (int t = 0; t < 32; ++t) {
            const float pt = __shfl_sync(0xffffffffu, p, t);
            const int pg = __shfl_sync(0xffffffffu, page, t);
            if (!__shfl_sync(0xffffffffu, (int)see, t))
                continue;
            const uint8_t *v = (const uint8_t *)c.v + (size_t)pg * c.v_stride[0] + (size_t)h * c.v_stride[1] +
                               (size_t)((j0 + t) % c.block) * c.v_stride[2];
            const float w = pt * c.v_scale[(size_t)pg * c.kv_heads + h];
            for (int d = 0; d < D / 64; ++d) {
                const float2 x2 = decode2(*(const uint16_t *)(v + d * 64 + lane * 2), c.code);
                o[2 * d] += w * x2.x;
                o[2 * d + 1] += w * x2.y;
            }
        }
    }
    for (int d = 0; d < D / 64; ++d) {
        __nv_bfloat16 *dst = a.out + r * D + d * 64 + lane * 2;
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        dst[0] = __float2bfloat16(o[2 * d] * inv);
        dst[1] = __float2bfloat16(o[2 * d + 1] * inv);
    }
    if (lane == 0)
        a.lse[r] = l > 0.0f || l != l ? m + logf(l) : -INFINITY;
}

// One warp per 32 tokens of a sequence and head, a lane per token, all rows.
__global__ void __launch_bounds__(128) weigh_kernel(const AttendArgs a, int chunks)
{
    __shared__ float sq[4][128];
    const spec_cache &c = a.c;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, D = c.dim, G = a.heads / c.kv_heads;
    const long long u = (long long)blockIdx.x * 4 + wid;
    if (u >= (long long)c.batch * c.kv_heads * chunks)
        return;
    const int j = (int)(u % chunks) * 32 + lane;
    const int h = (int)(u / chunks % c.kv_heads), b = (int)(u / chunks / c.kv_heads);
    const Seq s = sequence(c, a.lengths, a.f.num_new, a.n, b, true);
    if (!s.ok && lane == 0)
        report(a.status, SPEC_STATUS_BAD_LENGTH);
    const int page = j < s.len ? page_of(c, b, j / c.block) : -1;
    if (j < s.len && page < 0)
        report(a.status, SPEC_STATUS_BAD_PAGE);
    float *q = sq[wid], sum = 0.0f;
    for (int i = 0; i < s.m; ++i)
        for (int g = 0; g < G; ++g) {
            const int H = h * G + g;
            __syncwarp();
            for (int d = lane; d < D; d += 32)
                q[d] = __bfloat162float(a.q[b * a.q_stride[0] + i * a.q_stride[1] + H * a.q_stride[2] + d]);
            __syncwarp();
            const float lse = a.lse_in[((size_t)b * a.n + i) * a.heads + H];
            const float pos_q = a.f.slopes ? query_position(a, b, h, s.len - s.m + i) : 0.0f;
            if (page >= 0 && lse != -INFINITY && sees(a, s, b, i, j))
                sum += expf(score(a, q, page, h, j % c.block, a.f.slopes ? a.f.slopes[H] : 0.0f, pos_q, j) - lse);
        }
    if (page >= 0)
        a.weights[((size_t)page * c.kv_heads + h) * c.block + j % c.block] += sum;
}

spec_status check_call(const spec_cache *cache, const int32_t *lengths, const void *q, const int64_t q_stride[3],
                       int n, int heads, const spec_cache_form *form, const uint32_t *status)
{
    const spec_status st = check_cache(cache);
    if (st != SPEC_OK)
        return st;
    if (n < 0 || n > INT_MAX / 2 || heads < 1 || heads % cache->kv_heads || !form || form->window < 0 ||
        !(form->softcap >= 0.0f) || !(form->scale - form->scale == 0.0f) || !(form->softcap - form->softcap == 0.0f) ||
        (form->parent && n > SPEC_MAX_TREE_NODES))
        return SPEC_ERR_INVALID_ARG;
    if ((long long)n * heads > INT_MAX / 2)
        return SPEC_ERR_UNSUPPORTED;
    if (cache->batch == 0 || n == 0)
        return SPEC_OK;
    if (!q || !q_stride || ((uintptr_t)q & 15u) || bad4(lengths, true) || bad4(form->slopes, false) ||
        bad4(form->prefix, false) || bad4(form->parent, false) || bad4(form->num_new, false) || bad4(status, false))
        return SPEC_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
        if (q_stride[i] & 7)
            return SPEC_ERR_INVALID_ARG;
    return SPEC_OK;
}

AttendArgs make_args(const spec_cache *cache, const int32_t *lengths, const void *q, const int64_t q_stride[3], int n,
                     int heads, const spec_cache_form *form, uint32_t *status)
{
    AttendArgs a{};
    a.c = *cache;
    a.f = *form;
    a.lengths = lengths;
    a.q = (const __nv_bfloat16 *)q;
    for (int i = 0; i < 3; ++i)
        a.q_stride[i] = q_stride[i];
    a.n = n;
    a.heads = heads;
    a.status = status;
    return a;
}

}  // namespace

extern "C" {

spec_status spec_cache_attend_workspace(const spec_cache *cache, int n, int heads, int64_t *bytes)
{
    const spec_status st = check_cache(cache);
    if (st != SPEC_OK)
        return st;
    if (!bytes || n < 0 || heads < 1 || heads % cache->kv_heads)
        return SPEC_ERR_INVALID_ARG;
    *bytes = 0;
    return SPEC_OK;
}

spec_status spec_cache_attend(const spec_cache *cache, const int32_t *lengths, const void *q,
                              const int64_t q_stride[3], int n, int heads, const spec_cache_form *form, void *out,
                              float *lse, void *workspace, int64_t workspace_bytes, uint32_t *status, void *stream)
{
    NvtxScope nvtx("spec_cache_attend");
    spec_status st = check_call(cache, lengths, q, q_stride, n, heads, form, status);
    if (st != SPEC_OK || cache->batch == 0 || n == 0)
        return st;
    int64_t need = 0;
    st = spec_cache_attend_workspace(cache, n, heads, &need);
    if (st != SPEC_OK)
        return st;
    if (!out || ((uintptr_t)out & 15u) || bad4(lse, true) || workspace_bytes < need ||
        (need && !workspace) || ((uintptr_t)workspace & 15u))
        return SPEC_ERR_INVALID_ARG;
    AttendArgs a = make_args(cache, lengths, q, q_stride, n, heads, form, status);
    a.out = (__nv_bfloat16 *)out;
    a.lse = lse;
    const long long rows = (long long)cache->batch * n * heads;
    if (rows / 4 >= INT_MAX)
        return SPEC_ERR_UNSUPPORTED;
    attend_kernel<<<(unsigned)((rows + 3) / 4), 128, 0, (cudaStream_t)stream>>>(a);
    return launched();
}

spec_status spec_cache_weigh(const spec_cache *cache, const int32_t *lengths, const void *q,
                             const int64_t q_stride[3], int n, int heads, const spec_cache_form *form,
                             const float *lse, float *weights, uint32_t *status, void *stream)
{
    NvtxScope nvtx("spec_cache_weigh");
    const spec_status st = check_call(cache, lengths, q, q_stride, n, heads, form, status);
    if (st != SPEC_OK || cache->batch == 0 || n == 0)
        return st;
    if (bad4(lse, true) || bad4(weights, true))
        return SPEC_ERR_INVALID_ARG;
    AttendArgs a = make_args(cache, lengths, q, q_stride, n, heads, form, status);
    a.lse_in = lse;
    a.weights = weights;
    const int chunks = (cache->max_blocks * cache->block + 31) / 32;
    const long long warps = (long long)cache->batch * cache->kv_heads * chunks;
    if (warps / 4 >= INT_MAX)
        return SPEC_ERR_UNSUPPORTED;
    weigh_kernel<<<(unsigned)((warps + 3) / 4), 128, 0, (cudaStream_t)stream>>>(a, chunks);
    return launched();
}

}  // extern "C"
