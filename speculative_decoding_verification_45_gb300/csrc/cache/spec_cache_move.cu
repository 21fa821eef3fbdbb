// spec_cache_move.cu -- writing tokens into the 8-bit key/value cache and
// moving the kept ones out of it (spec_cache_append, spec_cache_evict).

#include <cooperative_groups.h>

#include <algorithm>

#include "spec_cache.cuh"

using namespace specc;
namespace cg = cooperative_groups;

namespace {

// ===========================================================================
// Append
// ===========================================================================
// One unit is one block of one sequence, head and side (keys or values): its
// scale depends on nothing else.  The unit's new values are read once, kept in
// registers as 8-value chunks (kChunks a thread) while their largest magnitude is
// found, and written as codes.  T threads serve a unit: a warp for the few tokens
// of a round, 256 threads for a prompt's whole blocks.
constexpr int kAppendThreads = 256;
constexpr int kAppendSmall = 16;  // new tokens up to which a warp's registers hold a unit (8 chunks a lane)

struct AppendArgs {
    spec_cache c;
    const int32_t *lengths, *num_new, *positions;
    const void *x[2];
    int64_t stride[2][3];
    int n, blocks;  // blocks a sequence may touch
    uint32_t units;
    uint32_t *status;
};

template <typename X> struct Chunk;
template <> struct Chunk<__nv_bfloat16> {
    uint4 raw;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool aligned)
    {
        if (aligned) {
            raw = __ldg((const uint4 *)p);
        } else {
            const unsigned short *s = (const unsigned short *)p;
            raw = make_uint4(s[0] | (uint32_t)s[1] << 16, s[2] | (uint32_t)s[3] << 16, s[4] | (uint32_t)s[5] << 16,
                             s[6] | (uint32_t)s[7] << 16);
        }
    }
    __device__ __forceinline__ float2 two(int i) const
    {
        const uint32_t w = i == 0 ? raw.x : i == 1 ? raw.y : i == 2 ? raw.z : raw.w;
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ __forceinline__ float largest() const  // magnitude; not finite if a value is not
    {
        uint32_t m = max_halves(max_halves(raw.x & 0x7fff7fffu, raw.y & 0x7fff7fffu),
                                max_halves(raw.z & 0x7fff7fffu, raw.w & 0x7fff7fffu));
        m = max(m & 0xffffu, m >> 16);
        return __uint_as_float(m << 16);
    }
};
template <> struct Chunk<float> {
    float4 lo, hi;
    __device__ __forceinline__ void load(const float *p, bool aligned)
    {
        if (aligned) {
            lo = __ldg((const float4 *)p);
            hi = __ldg((const float4 *)p + 1);
        } else {
            lo = make_float4(p[0], p[1], p[2], p[3]);
            hi = make_float4(p[4], p[5], p[6], p[7]);
        }
    }
    __device__ __forceinline__ float2 two(int i) const
    {
        return i == 0 ? make_float2(lo.x, lo.y) : i == 1 ? make_float2(lo.z, lo.w)
               : i == 2 ? make_float2(hi.x, hi.y) : make_float2(hi.z, hi.w);
    }
    __device__ __forceinline__ float largest() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // the bits of magnitudes order as they do, and NaN above them
            m = max(m, max(__float_as_uint(two(i).x) & 0x7fffffffu, __float_as_uint(two(i).y) & 0x7fffffffu));
        return __uint_as_float(m);
    }
};

template <typename X, int T, int kChunks, int CODE>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a)
{
    constexpr int kUnits = kAppendThreads / T;  // units of a CTA
    const spec_cache &c = a.c;
    const int sub = threadIdx.x / T, t = threadIdx.x % T;
    // 32-bit quotients: in 64 bits they were half of the kernel's instructions
    const uint32_t u = blockIdx.x * kUnits + sub;
    const bool here = u < a.units;
    const uint32_t u1 = here ? u : 0, u2 = (u1 >> 1) / (uint32_t)c.kv_heads, u3 = u2 / (uint32_t)a.blocks;
    const int side = (int)(u1 & 1), h = (int)((u1 >> 1) - u2 * c.kv_heads), k = (int)(u2 - u3 * a.blocks), b = (int)u3;
    const Seq s = sequence(c, a.lengths, a.num_new, a.n, b, false);
    if (here && t == 0 && !s.ok && k == 0 && side == 0 && h == 0)
        report(a.status, SPEC_STATUS_BAD_LENGTH);
    const int P = c.block, blk = s.len / P + k;
    const long long start = (long long)blk * P;
    const int old = max(0, (int)((long long)s.len - start));             // tokens that the block holds
    const int put = (int)min((long long)P, (long long)s.len + s.m - start) - old;  // tokens to write
    bool live = here && s.ok && put > 0;
    int page = -1;
    if (live) {
        page = page_of(c, b, blk);
        if (page < 0 && t == 0)
            report(a.status, SPEC_STATUS_BAD_PAGE);
        live = page >= 0;
    }
    const int per = c.dim / 8;  // chunks of a token: 8 or 16
    const int shift = c.dim == 64 ? 3 : 4;
    const int todo = live ? put * per : 0;
    const int i0 = (int)(start + old - s.len);  // index of the first token of this block among the new ones
    const X *src = (const X *)a.x[side] + (size_t)b * a.stride[side][0] + (size_t)h * a.stride[side][2];
    const bool aligned = (((uintptr_t)a.x[side] | (uintptr_t)(a.stride[side][0] * sizeof(X)) |
                           (uintptr_t)(a.stride[side][1] * sizeof(X)) | (uintptr_t)(a.stride[side][2] * sizeof(X))) &
                          15u) == 0;
    Chunk<X> x[kChunks];
    float amax = 0.0f;
    bool odd = false;  // a value is not finite
    // a thread's chunks are the same part of every (T / per)-th token
    const int token = t >> shift, d = (t & (per - 1)) * 8, step = T >> shift;
    {
        const X *p = src + (int64_t)(i0 + token) * a.stride[side][1] + d;
        const int64_t next = (int64_t)step * a.stride[side][1];
#pragma unroll
        for (int j = 0; j < kChunks; ++j, p += next)
            if (t + j * T < todo)
                x[j].load(p, aligned);
    }
    float *scale = (side ? c.v_scale : c.k_scale) + (size_t)max(page, 0) * c.kv_heads + h;
    const float had = live && old ? *scale : 0.0f;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        if (t + j * T < todo) {
            const float most = x[j].largest();
            if (isfinite(most)) {
                amax = fmaxf(amax, most);
            } else {
                odd = true;
                for (int i = 0; i < 4; ++i) {
                    const float2 v = x[j].two(i);
                    amax = isfinite(v.x) ? fmaxf(amax, fabsf(v.x)) : amax;
                    amax = isfinite(v.y) ? fmaxf(amax, fabsf(v.y)) : amax;
                }
            }
        }
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    if (T > 32) {
        __shared__ float part[kAppendThreads / 32];
        if ((threadIdx.x & 31) == 0)
            part[threadIdx.x >> 5] = amax;
        __syncthreads();  // also: every thread has read the old scale
#pragma unroll
        for (int w = 0; w < kAppendThreads / 32; ++w)
            amax = fmaxf(amax, part[w]);
    } else {
        __syncwarp();
    }
    if (!live)
        return;
    const float now = fmaxf(scale_for(amax, CODE), had);
    const int64_t *cs = side ? c.v_stride : c.k_stride;
    uint8_t *dst = (uint8_t *)(side ? c.v : c.k) + (size_t)page * cs[0] + (size_t)h * cs[1];
    const auto write = [&](auto encode) {
        uint8_t *p = dst + (int64_t)(old + token) * cs[2] + d;
        const int64_t next = (int64_t)step * cs[2];
#pragma unroll
        for (int j = 0; j < kChunks; ++j, p += next) {
            if (t + j * T < todo) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = encode(x[j].two(i));
                *(uint2 *)p = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
            }
        }
    };
    const Divider over(now);
    if (over.exact && !odd)
        write([&](float2 v) -> uint32_t { return encode2_finite(v.x * over.inv, v.y * over.inv, CODE); });
    else
        write([&](float2 v) -> uint32_t { return encode2(over(v.x), over(v.y), CODE); });
    if (old && now != had) {  // the block's scale grew: its older codes move to the new one
        const Mover move(had / now);
        for (int q = t; q < old * per; q += T) {
            uint2 *p = (uint2 *)(dst + (size_t)(q >> shift) * cs[2] + (q & (per - 1)) * 8);
            const uint2 w = *p;
            *p = make_uint2(move(w.x, CODE), move(w.y, CODE));
        }
    }
    if (t == 0)
        *scale = now;
    if (side == 0 && c.positions)
        for (int q = t; q < put; q += T)
            c.positions[((size_t)page * c.kv_heads + h) * P + old + q] =
                a.positions ? a.positions[(size_t)b * a.n + i0 + q] : s.len + i0 + q;
}

// ===========================================================================
// Evict
// ===========================================================================
// Two kernels: one CTA or cluster per (sequence, head) finds the kept indices,
// then one CTA per block of kept tokens moves them.  Sources and destinations share no
// page, so the moves need no order.
constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kDigits = 2048;  // 11 bits at a time: 3 rounds
constexpr int kMoveThreads = 256;

struct EvictArgs {
    spec_cache c;
    const int32_t *lengths, *out_table;
    float *weights;
    int64_t out_stride;
    int32_t *out_lengths, *out_index;
    int keep, recent;
    uint32_t *status;
};

// Weight to an unsigned key of the same order: NaN lowest, both zeros alike.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w)
        return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Keys of the tokens j, j + step, ... below end, 0 where there is none.  All their pages are asked for at once, then all
// their weights: taken one by one, the two latencies were a third of the kernel's time.
constexpr int kAhead = 8;
__device__ __forceinline__ void load_keys(const EvictArgs &a, int b, int h, int log_p, int j, int step, int end,
                                          uint32_t (&key)[kAhead])
{
    int page[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        page[i] = j + i * step < end ? page_of(a.c, b, (j + i * step) >> log_p) : -1;
    float w[kAhead];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        bad = bad || (page[i] < 0 && j + i * step < end);
    if (bad)
        report(a.status, SPEC_STATUS_BAD_PAGE);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        w[i] = page[i] < 0 ? __int_as_float(0x7fffffff)
                           : a.weights[(((size_t)page[i] * a.c.kv_heads + h) << log_p) + ((j + i * step) & ((1 << log_p) - 1))];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        key[i] = weight_key(w[i]);
}

// The (keep - recent)-th largest key is found 11 bits at a time from the top (a
// histogram of the keys that share the bits found so far); then each warp counts
// its stretch of tokens above the key and equal to it, and a second walk writes
// the indices in order.  The keys are kept in shared memory where they fit
// (`staged`), else read again from L2.  Keys equal to zero's, the one value that
// repeats in earnest (tokens that no query looked at), are counted by ballot.
// A cluster's CTAs take a stretch of the tokens each; every one of them adds the
// same histograms up and comes to the same digits.
template <int CS> __global__ void __launch_bounds__(kSelectThreads) select_kernel(const EvictArgs a, int staged)
{
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = CS > 1 ? (int)cluster.block_rank() : 0;
    asm volatile("griddepcontrol.launch_dependents;");  // the moving CTAs may take their places, and wait there
    const auto meet = [&] {
        if (CS > 1)
            cluster.sync();
        else
            __syncthreads();
    };
    extern __shared__ uint32_t keys[];
    __shared__ alignas(8) uint32_t hist[kDigits];
    __shared__ uint32_t warp_sum[kSelectWarps];
    __shared__ int count[2][kSelectWarps];
    __shared__ uint32_t found, left;
    __shared__ int len0, sum[2];
    const spec_cache &c = a.c;
    const int unit = blockIdx.x / CS, h = unit % c.kv_heads, b = unit / c.kv_heads, log_p = 31 - __clz(c.block);
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, all_tid = rank * kSelectThreads + tid;
    const Seq s = sequence(c, a.lengths, nullptr, 0, b, true);
    if (all_tid == 0 && h == 0 && !s.ok)
        report(a.status, SPEC_STATUS_BAD_LENGTH);
    int len = s.len;
    if (CS > 1) {  // one length for the cluster, whatever becomes of the array
        if (tid == 0)
            len0 = len;
        cluster.sync();
        len = *cluster.map_shared_rank(&len0, 0);
    }
    int32_t *index = a.out_index + ((size_t)b * c.kv_heads + h) * a.keep;
    for (int i = min(len, a.keep) + all_tid; i < a.keep; i += CS * kSelectThreads)
        index[i] = -1;
    const int all = len - a.recent, want = a.keep - a.recent;  // candidates; want < all where it matters
    if (len <= a.keep) {
        for (int i = all_tid; i < len; i += CS * kSelectThreads)
            index[i] = i;
    } else {
        for (int i = all_tid; i < a.recent; i += CS * kSelectThreads)
            index[want + i] = all + i;
    }
    if (len <= a.keep || want == 0) {
        if (CS > 1)
            cluster.sync();  // len0 is read
        return;
    }
    // this CTA's candidates: [begin, begin + cand)
    const int share = (all + CS - 1) / CS, begin = min(all, rank * share), cand = min(all, begin + share) - begin;
    const auto get = [&](int j, int step, int end, uint32_t (&key)[kAhead]) {
        if (!staged)
            return load_keys(a, b, h, log_p, begin + j, step, begin + end, key);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            key[i] = j + i * step < end ? keys[j + i * step] : 0;
    };
    const uint32_t zero = 0x80000000u;
    uint32_t prefix = 0, need = (uint32_t)want;  // rank of the wanted key among those that share `prefix`
    int shift = 21;
    for (int round = 0; round < 3; ++round) {
        const int bits = round < 2 ? 11 : 10;
        for (int i = tid; i < kDigits; i += kSelectThreads)
            hist[i] = 0;
        __syncthreads();
        const bool zeros = round == 0 || prefix == zero >> (shift + bits);  // zeros may be among those that share it
        for (int j0 = tid; j0 - tid < cand; j0 += kAhead * kSelectThreads) {
            uint32_t key[kAhead];
            if (round == 0)
                load_keys(a, b, h, log_p, begin + j0, kSelectThreads, begin + cand, key);
            else
                get(j0, kSelectThreads, cand, key);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int j = j0 + i * kSelectThreads;
                if (round == 0 && staged && j < cand)
                    keys[j] = key[i];
                const bool in = j < cand && (round == 0 || (key[i] >> (shift + bits)) == prefix);
                uint32_t *bin = &hist[(key[i] >> shift) & ((1u << bits) - 1)];
                const bool none = zeros && in && key[i] == zero;
                if (in && !none)
                    atomicAdd(bin, 1u);
                if (zeros) {
                    const uint32_t all = __ballot_sync(0xffffffffu, none);
                    if (none && lane == __ffs(all) - 1)
                        atomicAdd(bin, (uint32_t)__popc(all));
                }
            }
        }
        meet();
        // the digit where the count from the top reaches `need`: two bins a thread, top first
        uint32_t upper = 0, lower = 0;
#pragma unroll
        for (int r = 0; r < CS; ++r) {
            uint32_t *at = &hist[kDigits - 2 - 2 * tid];
            const uint2 two = *(const uint2 *)(CS > 1 ? cluster.map_shared_rank(at, r) : at);
            upper += two.y;
            lower += two.x;
        }
        uint32_t up = upper + lower;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, up, o);
            up += lane >= o ? y : 0;
        }
        if (lane == 31)
            warp_sum[wid] = up;
        __syncthreads();
        uint32_t ahead = lane < wid ? warp_sum[lane] : 0;
        ahead = __reduce_add_sync(0xffffffffu, ahead) + up - upper - lower;
        if (ahead < need && need <= ahead + upper + lower) {
            const bool second = need > ahead + upper;
            found = kDigits - 1 - 2 * tid - second;
            left = need - ahead - (second ? upper : 0);
        }
        meet();
        prefix = prefix << bits | found;
        need = left;
        shift -= round == 0 ? 11 : 10;
    }
    // tokens above the key `prefix` are all kept, of those equal to it the first `need`
    const int each = ((cand + kSelectWarps - 1) / kSelectWarps + 31) & ~31;
    const int lo = min(cand, wid * each), hi = min(cand, lo + each);
    int above = 0, equal = 0;
    for (int j = lo + lane; j < hi; j += kAhead * 32) {
        uint32_t key[kAhead];
        get(j, 32, hi, key);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            above += j + i * 32 < hi && key[i] > prefix;
            equal += j + i * 32 < hi && key[i] == prefix;
        }
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        count[0][wid] = above;
        count[1][wid] = equal;
    }
    __syncthreads();
    int at = __reduce_add_sync(0xffffffffu, lane < wid ? count[0][lane] : 0);
    int ties = __reduce_add_sync(0xffffffffu, lane < wid ? count[1][lane] : 0);
    if (CS > 1) {  // and the CTAs before this one
        if (wid == kSelectWarps - 1 && lane == 0) {
            sum[0] = at + above;
            sum[1] = ties + equal;
        }
        cluster.sync();
        for (int r = 0; r < rank; ++r) {
            const int *before = cluster.map_shared_rank(sum, r);
            at += before[0];
            ties += before[1];
        }
        cluster.sync();  // nobody leaves while its sums are read
    }
    int out = at + min(ties, (int)need);  // kept tokens before this warp's stretch
    const uint32_t below = (1u << lane) - 1;
    for (int j0 = lo; j0 < hi; j0 += kAhead * 32) {
        uint32_t key[kAhead];
        get(j0 + lane, 32, hi, key);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int j = j0 + i * 32 + lane;
            const bool eq = j < hi && key[i] == prefix;
            const uint32_t tie = __ballot_sync(0xffffffffu, eq);
            const bool take = (j < hi && key[i] > prefix) || (eq && ties + __popc(tie & below) < (int)need);
            const uint32_t took = __ballot_sync(0xffffffffu, take);
            if (take)
                index[out + __popc(took & below)] = begin + j;
            out += __popc(took);
            ties += __popc(tie);
        }
    }
}

template <int CODE> __global__ void __launch_bounds__(kMoveThreads, 6) move_kernel(const EvictArgs a, int blocks)
{
    __shared__ int from[kMaxBlock], row[kMaxBlock];  // source page of each token, -1: none
    __shared__ float had[2][kMaxBlock];              // its scales
    __shared__ long long off[2][kMaxBlock];          // where its codes lie, -1: nowhere
    const spec_cache &c = a.c;
    const int P = c.block, tid = threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for select_kernel
    const int k = blockIdx.x % blocks;
    const int h = (blockIdx.x / blocks) % c.kv_heads, b = blockIdx.x / blocks / c.kv_heads;
    const int to = a.out_table[(size_t)b * a.out_stride + k];
    const int kept = min(sequence(c, a.lengths, nullptr, 0, b, true).len, a.keep);
    const int n = min(P, kept - k * P);
    if (tid == 0 && h == 0 && k == 0)
        a.out_lengths[b] = kept;  // may be a.lengths: who reads it afterwards comes to the same
    if (n <= 0)
        return;
    if ((unsigned)to >= (unsigned)c.num_pages) {
        if (tid == 0)
            report(a.status, SPEC_STATUS_BAD_PAGE);
        return;
    }
    const int log_p = 31 - __clz(P);
    if (tid < n) {
        const int j = a.out_index[((size_t)b * c.kv_heads + h) * a.keep + k * P + tid];
        const int page = page_of(c, b, j >> log_p);
        if (page < 0)
            report(a.status, SPEC_STATUS_BAD_PAGE);
        from[tid] = page;
        row[tid] = j & (P - 1);
        off[0][tid] = page < 0 ? -1 : (long long)page * c.k_stride[0] + (long long)h * c.k_stride[1] + row[tid] * c.k_stride[2];
        off[1][tid] = page < 0 ? -1 : (long long)page * c.v_stride[0] + (long long)h * c.v_stride[1] + row[tid] * c.v_stride[2];
    }
    __syncthreads();
    // the codes are asked for before the scales that they may have to be changed by; half of the threads move keys, half
    // values, each the same 16 bytes of every few tokens
    const int shift = c.dim == 64 ? 2 : 3, side = tid >= kMoveThreads / 2, t = tid & (kMoveThreads / 2 - 1);
    const int d = (t & ((1 << shift) - 1)) * 16, step = (kMoveThreads / 2) >> shift;
    uint8_t *codes = (uint8_t *)(side ? c.v : c.k) + d;
    const int64_t *cs = side ? c.v_stride : c.k_stride;
    constexpr int kAtOnce = 4;  // loads in flight
    uint4 w[kAtOnce];
    const auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int i = i0 + k * step;
            const long long at = i < n ? off[side][i] : -1;
            w[k] = at >= 0 ? *(const uint4 *)(codes + at) : make_uint4(0, 0, 0, 0);
        }
    };
    load(t >> shift);
    if (tid < n) {
        const int page = from[tid];
        const size_t src = (size_t)max(page, 0) * c.kv_heads + h, dst = ((((size_t)to * c.kv_heads + h)) << log_p) + tid;
        const size_t at = (src << log_p) + row[tid];
        const float ks = page < 0 ? 0.0f : c.k_scale[src], vs = page < 0 ? 0.0f : c.v_scale[src];
        const float weight = page < 0 ? 0.0f : a.weights[at];
        const int position = page < 0 || !c.positions ? 0 : c.positions[at];
        had[0][tid] = ks;
        had[1][tid] = vs;
        a.weights[dst] = weight;
        if (c.positions)
            c.positions[dst] = position;
    }
    __syncthreads();
    float now[2] = {0.0f, 0.0f};
    for (int i = tid & 31; i < n; i += 32) {
        now[0] = fmaxf(now[0], had[0][i]);
        now[1] = fmaxf(now[1], had[1][i]);
    }
    // scales are positive: their bits order as they do
    now[0] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(now[0])));
    now[1] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(now[1])));
    // none of the block's tokens is cached: their codes are zeros, at the scale that append gives zeros
    now[0] = now[0] > 0.0f ? now[0] : 0x1p-100f;
    now[1] = now[1] > 0.0f ? now[1] : 0x1p-100f;
    if (tid < 2) {
        float *scale = tid ? c.v_scale : c.k_scale;
        scale[(size_t)to * c.kv_heads + h] = now[tid];
    }
    __shared__ float factor[2][kMaxBlock];  // 1: the codes stay
    if (tid < n) {
        factor[0][tid] = from[tid] < 0 ? 1.0f : had[0][tid] / now[0];
        factor[1][tid] = from[tid] < 0 ? 1.0f : had[1][tid] / now[1];
    }
    __syncthreads();
    uint8_t *out = codes + (size_t)to * cs[0] + (size_t)h * cs[1];
    for (int i0 = t >> shift; i0 < n; i0 += kAtOnce * step) {
        if (i0 != t >> shift)
            load(i0);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int i = i0 + k * step;
            if (i >= n)
                break;
            const float f = factor[side][i];
            if (f != 1.0f) {
                const Mover move(f);
                w[k] = make_uint4(move(w[k].x, CODE), move(w[k].y, CODE), move(w[k].z, CODE), move(w[k].w, CODE));
            }
            *(uint4 *)(out + (int64_t)i * cs[2]) = w[k];
        }
    }
}

template <typename X, int T, int kChunks> spec_status run_append(AppendArgs a, cudaStream_t stream)
{
    const long long units = (long long)a.c.batch * a.blocks * a.c.kv_heads * 2;
    const long long ctas = (units + kAppendThreads / T - 1) / (kAppendThreads / T);
    if (units > INT_MAX)
        return SPEC_ERR_UNSUPPORTED;
    a.units = (uint32_t)units;
    if (a.c.code == SPEC_E4M3)
        append_kernel<X, T, kChunks, SPEC_E4M3><<<(unsigned)ctas, kAppendThreads, 0, stream>>>(a);
    else
        append_kernel<X, T, kChunks, SPEC_E5M2><<<(unsigned)ctas, kAppendThreads, 0, stream>>>(a);
    return launched();
}

// Chunks a thread: as many as the unit's tokens (a block, or the new ones) need.  Fewer registers let more units
// be in flight.
template <typename X> spec_status choose_append(const AppendArgs &a, cudaStream_t s)
{
    const int chunks = a.c.dim / 8;
    if (a.n <= kAppendSmall) {
        const int each = (std::min(a.n, a.c.block) * chunks + 31) / 32;
        return each <= 2 ? run_append<X, 32, 2>(a, s) : each <= 4 ? run_append<X, 32, 4>(a, s) : run_append<X, 32, 8>(a, s);
    }
    const int each = (a.c.block * chunks + kAppendThreads - 1) / kAppendThreads;
    return each <= 2   ? run_append<X, kAppendThreads, 2>(a, s)
           : each <= 4 ? run_append<X, kAppendThreads, 4>(a, s)
                       : run_append<X, kAppendThreads, 8>(a, s);
}

}  // namespace

extern "C" {

spec_status spec_cache_append(const spec_cache *cache, const int32_t *lengths, const void *k, const void *v,
                              const int64_t k_stride[3], const int64_t v_stride[3], int n, spec_dtype dtype,
                              const int32_t *num_new, const int32_t *positions, uint32_t *status, void *stream)
{
    NvtxScope nvtx("spec_cache_append");
    spec_status st = check_cache(cache);
    if (st != SPEC_OK)
        return st;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16)
        return SPEC_ERR_UNSUPPORTED;
    if (n < 0 || n > INT_MAX / 2)
        return SPEC_ERR_INVALID_ARG;
    if (cache->batch == 0 || n == 0)
        return SPEC_OK;
    const uintptr_t mask = dtype == SPEC_F32 ? 3u : 1u;
    if (!k || !v || !k_stride || !v_stride || ((uintptr_t)k & mask) || ((uintptr_t)v & mask) ||
        bad4(lengths, true) || bad4(num_new, false) || bad4(positions, false) || bad4(status, false))
        return SPEC_ERR_INVALID_ARG;
    AppendArgs a;
    a.c = *cache;
    a.lengths = lengths;
    a.num_new = num_new;
    a.positions = positions;
    a.x[0] = k;
    a.x[1] = v;
    for (int i = 0; i < 3; ++i) {
        a.stride[0][i] = k_stride[i];
        a.stride[1][i] = v_stride[i];
    }
    a.n = n;
    a.blocks = (n + cache->block - 2) / cache->block + 1;
    a.status = status;
    const cudaStream_t s = (cudaStream_t)stream;
    return dtype == SPEC_F32 ? choose_append<float>(a, s) : choose_append<__nv_bfloat16>(a, s);
}

spec_status spec_cache_evict(const spec_cache *cache, const int32_t *lengths, float *weights, int keep, int recent,
                             const int32_t *out_table, int64_t out_stride, int32_t *out_lengths, int32_t *out_index,
                             uint32_t *status, void *stream)
{
    NvtxScope nvtx("spec_cache_evict");
    spec_status st = check_cache(cache);
    if (st != SPEC_OK)
        return st;
    if (keep < 1 || keep > INT_MAX / 2 || recent < 0 || recent > keep)
        return SPEC_ERR_INVALID_ARG;
    if (cache->batch == 0)
        return SPEC_OK;
    const int blocks = (keep + cache->block - 1) / cache->block;
    if (bad4(lengths, true) || bad4(weights, true) || bad4(out_table, true) || bad4(out_lengths, true) ||
        bad4(out_index, true) || bad4(status, false) || out_stride < blocks)
        return SPEC_ERR_INVALID_ARG;
    const long long heads = (long long)cache->batch * cache->kv_heads;
    if (heads * blocks > INT_MAX)
        return SPEC_ERR_UNSUPPORTED;
    EvictArgs a{*cache, lengths, out_table, weights, out_stride, out_lengths, out_index, keep, recent, status};
    const cudaStream_t s = (cudaStream_t)stream;
    const long long room = (long long)cache->max_blocks * cache->block;
    // few long sequences: clusters, as many CTAs as the SMs hold, of 8,192 tokens or more each (2 sequences of 100,000
    // tokens and 8 heads: 68 us against 171; 7 of 16,384: 45 against 47; pairs of 4,096 tokens each: 44 against 40)
    int log_cluster = 0;
    while (log_cluster < 3 && heads << (log_cluster + 1) <= 128 && room >= 8192ll << (log_cluster + 1))
        ++log_cluster;
    static constexpr void (*kSelect[])(EvictArgs, int) = {select_kernel<1>, select_kernel<2>, select_kernel<4>, select_kernel<8>};
    const auto select = kSelect[log_cluster];
    const int cluster = 1 << log_cluster;
    // shared memory for the keys of the longest sequence; up to 48 KB needs no opt-in
    const long long bytes = (room + cluster - 1) / cluster * 4;
    const int staged = bytes <= 200 * 1024;
    if (staged && bytes > 36 * 1024 &&
        cudaFuncSetAttribute((const void *)select, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) != cudaSuccess) {
        cudaGetLastError();
        return SPEC_ERR_CUDA;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(heads * cluster));
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = staged ? (size_t)bytes : 0;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1;
    if (cudaLaunchKernelEx(&cfg, select, a, staged) != cudaSuccess) {
        cudaGetLastError();
        return SPEC_ERR_CUDA;
    }
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(heads * blocks));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, cache->code == SPEC_E4M3 ? move_kernel<SPEC_E4M3> : move_kernel<SPEC_E5M2>, a, blocks) !=
        cudaSuccess) {
        cudaGetLastError();
        return SPEC_ERR_CUDA;
    }
    return SPEC_OK;
}

}  // extern "C"
