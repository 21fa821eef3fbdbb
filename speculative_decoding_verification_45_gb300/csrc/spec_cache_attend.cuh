// spec_cache_attend.cuh -- attention over the 8-bit key/value cache on the
// tensor cores, and the attention weight that each cached token received.
// include/spec_verify.h states the operations.
//
// The matrix products take the codes as they lie in memory: kind::f8f6f4
// multiplies 8-bit floats, so keys and values go from HBM through TMA into
// shared memory and from there into tcgen05.mma, with no conversion between.
// What multiplies them is split so that 8 bits lose nothing:
//   q    a bf16 value (8-bit significand), scaled by a power of two per row, is
//        exactly the sum of two e4m3 values (4 bits each; the remainder after
//        rounding to 4 bits needs no more than 4), down to 2^-10 of the row's
//        largest element;
//   p    exp(x - ..) scaled per tile and row so that the largest lies in
//        [128, 256), as the sum of two e4m3 values: 2^-8 relative, the rounding
//        of a bf16 weight.
// Each product is issued once per term into the same accumulator.
//
// Tokens are the M side (128 per tile), query rows the N side: a decode step
// has few rows (new tokens x query heads per key head), which would fill a
// fraction of an M = 128 tile, while N may be 16, 32 or 64.  So
//   S^T [128 tokens, NT rows] = K [128, D] Q^T        (K is K-major as stored)
//   O^T [D, NT rows]          = V^T [D, 128] P^T      (V is M-major as stored)
// and a thread of the softmax owns one token and NT / 2 rows, with every lane
// busy whatever the number of rows.
#ifndef SPEC_CACHE_ATTEND_CUH
#define SPEC_CACHE_ATTEND_CUH

#include <cuda.h>

#include "spec_cache.cuh"

namespace specc {

struct AttendArgs {
    spec_cache c;
    spec_cache_form f;
    const int32_t *lengths;
    const __nv_bfloat16 *q;
    int64_t q_stride[3];
    int n, heads, group;   // group: query heads per key/value head
    int row_tiles;         // ceil(n * group / NT)
    __nv_bfloat16 *out;
    float *lse;
    const float *lse_in;
    float *weights;
    float *part;           // [2 * CTAs][NT][D] partial sums, then [2 * CTAs][NT] (total, base)
    float2 *part_sum;
    int4 *joins;           // [CTAs]: (first CTA or -1, sequence, head, row tile)
    uint32_t *status;
};

constexpr int kTile = 128;
constexpr int kMaxNodes = SPEC_MAX_TREE_NODES;
constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok;
}
// Waits for a phase, a bounded number of tries.  When they run out `dead` is set
// and every later wait returns at once: control flow stays the same for all
// threads, so the CTA runs to its end (with results that the status marks bad).
constexpr uint32_t kTries = 1u << 22;
__device__ __forceinline__ void mbar_wait(uint64_t *bar, uint32_t parity, volatile int *dead)
{
    if (mbar_try(bar, parity))
        return;
    for (uint32_t i = 0; i < kTries; ++i) {
        if (mbar_try(bar, parity) || *dead)
            return;
    }
    *dead = 1;
}

// After a wait ran out: copies and products in flight end before the CTA's memory is given back.
template <int ST>
__device__ __forceinline__ void drain(uint64_t *full, uint32_t issued, volatile int *dead, uint32_t *status)
{
    if (!*dead)
        return;
    for (uint32_t i = 0; i < ST && i < issued; ++i) {
        const uint32_t parity = ((issued - 1 - i) / ST) & 1;  // of the stage's last copy
        for (uint32_t k = 0; k < 4096 && !mbar_try(&full[i], parity); ++k)
            ;
    }
    report(status, SPEC_STATUS_INTERNAL);
}
__device__ __forceinline__ void tc_commit(uint64_t *bar);
__device__ __forceinline__ void drain_products(uint64_t *bar, volatile int *dead)
{
    if (!*dead || (threadIdx.x & 31))
        return;
    tc_commit(bar);
    for (uint32_t k = 0; k < 4096 && !mbar_try(bar, 0); ++k)
        ;
}

template <int N> __device__ __forceinline__ void named_barrier(int id)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
}

__device__ __forceinline__ void tma_load(const CUtensorMap *map, void *dst, uint64_t *bar, int d, int row, int head, int page)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, "
                 "%6}], [%2];" ::"r"(smem_u32(dst)),
                 "l"(map), "r"(smem_u32(bar)), "r"(d), "r"(row), "r"(head), "r"(page)
                 : "memory");
}
__device__ __forceinline__ void bulk_load(const void *src, void *dst, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void copy4(const void *src, void *dst)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t *bar)  // when this thread's earlier copies are done
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
                 : "memory");
}
template <int N> struct TmemLoad;
template <> struct TmemLoad<8> {
    static __device__ __forceinline__ void go(uint32_t a, float *r)
    {
        uint32_t *u = (uint32_t *)r;
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                     : "r"(a));
    }
};
template <> struct TmemLoad<16> {
    static __device__ __forceinline__ void go(uint32_t a, float *r)
    {
        uint32_t *u = (uint32_t *)r;
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                     : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
                       "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
                     : "r"(a));
    }
};
template <> struct TmemLoad<32> {
    static __device__ __forceinline__ void go(uint32_t a, float *r)
    {
        TmemLoad<16>::go(a, r);
        TmemLoad<16>::go(a + 16, r + 16);
    }
};
// The registers of earlier loads are valid after this; they pass through it so that no use moves ahead.
template <int N> __device__ __forceinline__ void tmem_wait(float *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+f"(r[i]));
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Shared-memory matrix descriptor.  swizzle: 0 none, 2 128-byte, 4 64-byte.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint64_t swizzle)
{
    return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)((lbo >> 4) & 0x3fff) << 16 | (uint64_t)((sbo >> 4) & 0x3fff) << 32 |
           1ull << 46 | swizzle << 61;
}
// Instruction descriptor: float accumulator, M = 128; a_code 0 e4m3, 1 e5m2; B is e4m3.
__device__ __forceinline__ uint32_t instr_desc(int nt, int a_code, bool a_mn, bool b_mn)
{
    return 1u << 4 | (uint32_t)a_code << 7 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 | (uint32_t)(nt >> 3) << 17 |
           (uint32_t)(kTile >> 4) << 24;
}

// ---------------------------------------------------------------------------
// Work: which tiles a row tile of a sequence reads
// ---------------------------------------------------------------------------
// Tiles [0, head_tiles) (a prefix before the window), then [low, low + count - head_tiles).
struct Unit {
    int len, m, first, prefix;
    int i0, i1;  // queries of the row tile
    int head_tiles, low, count;
    __device__ __forceinline__ int tile(int x) const { return x < head_tiles ? x : x - head_tiles + low; }
};

__device__ __forceinline__ Unit unit_for(const AttendArgs &a, int b, int i0, int i1)
{
    Unit u;
    const Seq s = sequence(a.c, a.lengths, a.f.num_new, a.n, b, true);
    u.len = s.len;
    u.m = s.m;
    u.first = s.len - s.m;
    u.prefix = a.f.prefix ? min(max(a.f.prefix[b], 0), s.len) : 0;
    u.i0 = i0;
    u.i1 = min(i1, s.m - 1);
    u.head_tiles = u.low = u.count = 0;
    if (u.i0 > u.i1)
        return u;
    const int ptiles = (u.prefix + kTile - 1) / kTile;
    if (a.f.window > 0)
        u.low = (int)(max(0ll, (long long)u.first + u.i0 - a.f.window + 1) / kTile);
    u.head_tiles = min(ptiles, u.low);
    u.count = u.head_tiles + max((u.first + u.i1) / kTile + 1, ptiles) - u.low;
    return u;
}

template <int NT> __device__ __forceinline__ Unit row_unit(const AttendArgs &a, int b, int rt)
{
    return unit_for(a, b, rt * NT / a.group, (rt * NT + NT - 1) / a.group);
}

// Every token of the tile at j0 is seen by every query of the unit.
__device__ __forceinline__ bool interior(const AttendArgs &a, const Unit &u, int j0)
{
    const long long last = (long long)j0 + kTile - 1;
    if (last >= u.len)
        return false;
    if (last < u.prefix)
        return true;
    return last <= (a.f.parent ? u.first - 1 : u.first + u.i0) &&
           (a.f.window <= 0 || (long long)j0 > (long long)u.first + u.i1 - a.f.window);
}

// The tiles of all units in order, cut into equal stretches, one per CTA.  A
// unit without a tile counts as one, so that its rows are written.
struct Range {
    long long begin, end, each;
    int b;
    long long skip;  // tiles of sequence b before `begin`
};

// COST(b): tiles of sequence b.  All threads of the CTA call this.
template <int THREADS, typename Cost> __device__ __forceinline__ Range find_range(const AttendArgs &a, Cost cost)
{
    __shared__ long long warp_sum[THREADS / 32];
    __shared__ Range range;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, B = a.c.batch;
    long long total = 0;
    if (tid == 0)
        range.begin = range.end = 0;
    for (int pass = 0; pass < 2; ++pass) {
        long long seen = 0, each = 0, begin = 0;
        if (pass == 1) {
            each = (total + gridDim.x - 1) / gridDim.x;
            begin = (long long)blockIdx.x * each;
        }
        for (int b0 = 0; b0 < B; b0 += THREADS) {
            const int b = b0 + tid;
            const long long mine = b < B ? cost(b) : 0;
            long long up = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, up, o);
                up += lane >= o ? y : 0;
            }
            if (lane == 31)
                warp_sum[wid] = up;
            __syncthreads();
            long long all = 0;
            for (int w = 0; w < THREADS / 32; ++w) {
                all += warp_sum[w];
                up += w < wid ? warp_sum[w] : 0;
            }
            if (pass == 1 && begin < total && b < B && seen + up - mine <= begin && begin < seen + up) {
                range.begin = begin;
                range.end = min(begin + each, total);
                range.each = each;
                range.b = b;
                range.skip = begin - (seen + up - mine);
            }
            seen += all;
            __syncthreads();
        }
        total = seen;
    }
    return range;
}

// ---------------------------------------------------------------------------
// What both kernels keep in shared memory for the columns (query rows) of a row tile
// ---------------------------------------------------------------------------
template <int NT> struct Columns {
    float factor[NT];  // of the accumulator, times the token's scale: the score, in units of log2 (of softcap with one)
    float base[NT];    // attend: the exponent's reference; weigh: the row's lse, in units of log2
    float slope[NT];   // times log2(e)
    float pos[NT];
    int query[NT];     // its query, -1: none
    uint32_t kin[NT][kMaxNodes / 32];
    int up[kMaxNodes];
};

// Rows of a row tile into shared memory as two e4m3 terms, 128- or 64-byte
// swizzled, and the columns' constants.  Called by 256 threads (t), which have
// met at a barrier after the last use of either; ends without one.
template <int D, int NT>
__device__ __forceinline__ void load_queries(const AttendArgs &a, const Unit &u, int b, int h, int rt, bool tree, uint8_t *q,
                                             Columns<NT> &col, int t)
{
    constexpr int kLanes = D / 8, kRows = 256 / kLanes;
    const int d = t % kLanes;
    if (tree && a.f.parent)
        for (int k = t; k < u.m; k += 256) {
            const int up = k > 0 ? a.f.parent[(size_t)b * a.n + k] : -1;
            if (k > 0 && (unsigned)up >= (unsigned)k)
                report(a.status, SPEC_STATUS_BAD_TREE);
            col.up[k] = (unsigned)up < (unsigned)k ? up : -1;
        }
#pragma unroll
    for (int r0 = 0; r0 < NT; r0 += kRows) {
        const int c = r0 + t / kLanes;
        if (kRows > NT && c >= NT)
            continue;  // whole warps: a warp holds 2 or 4 rows
        const int r = rt * NT + c, i = r / a.group, H = h * a.group + r % a.group;
        const bool live = i <= u.i1;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (live)
            w = __ldg((const uint4 *)(a.q + (size_t)b * a.q_stride[0] + (size_t)i * a.q_stride[1] +
                                      (size_t)H * a.q_stride[2] + d * 8));
        float x[8];
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(ww[e] << 16);
            x[2 * e + 1] = __uint_as_float(ww[e] & 0xffff0000u);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            amax = isfinite(x[e]) ? fmaxf(amax, fabsf(x[e])) : amax;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        // the row's power of two: its largest element becomes [128, 256)
        const int ex = amax > 0.0f ? max((int)(__float_as_uint(amax) >> 23), 16) - 7 : 127;  // biased
        const float inv = __uint_as_float((uint32_t)(254 - ex) << 23);
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float y[4], z[4];
            uint32_t code[2], rest[2];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                y[k] = x[4 * e + k] * inv;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                code[k] = encode2(y[2 * k], y[2 * k + 1], SPEC_E4M3);
                const float2 back = decode2((uint16_t)code[k], SPEC_E4M3);
                z[2 * k] = y[2 * k] - back.x;
                z[2 * k + 1] = y[2 * k + 1] - back.y;
                rest[k] = encode2(z[2 * k], z[2 * k + 1], SPEC_E4M3);
            }
            hi[e] = code[0] | code[1] << 16;
            lo[e] = rest[0] | rest[1] << 16;
        }
        const int at = c * D + ((d * 8) ^ (D == 128 ? (c & 7) << 4 : ((c >> 1) & 3) << 4));
        *(uint2 *)(q + at) = make_uint2(hi[0], hi[1]);
        *(uint2 *)(q + NT * D + at) = make_uint2(lo[0], lo[1]);
        if (d == 0) {
            const float row = __uint_as_float((uint32_t)ex << 23) * a.f.scale;
            col.factor[c] = a.f.softcap > 0.0f ? row / a.f.softcap : row * kLog2e;
            col.query[c] = live ? i : -1;
            if (a.f.slopes) {
                const int at_j = u.first + i;
                float p = (float)at_j;
                if (live && a.c.positions) {
                    const int page = page_of(a.c, b, at_j / a.c.block);
                    p = page < 0 ? 0.0f
                                 : (float)a.c.positions[((size_t)page * a.c.kv_heads + h) * a.c.block + at_j % a.c.block];
                }
                col.pos[c] = p;
                col.slope[c] = live ? a.f.slopes[H] * kLog2e : 0.0f;
            }
        }
    }
}

// The ancestors of each column's query, after a barrier behind load_queries.
template <int NT> __device__ __forceinline__ void mark_kin(const Unit &u, Columns<NT> &col, int t)
{
    if (t < NT) {
        for (int w = 0; w < kMaxNodes / 32; ++w)
            col.kin[t][w] = 0;
        for (int k = col.query[t]; k >= 0; k = col.up[k])
            col.kin[t][k >> 5] |= 1u << (k & 31);
    }
}

// Does column c's query see token j (cached)?
template <int NT>
__device__ __forceinline__ bool sees(const AttendArgs &a, const Unit &u, const Columns<NT> &col, int c, int j)
{
    const int i = col.query[c], t = j - u.first;
    bool see = t <= i;
    if (a.f.parent && t >= 0 && t < u.m)
        see = (col.kin[c][t >> 5] >> (t & 31)) & 1;
    if (a.f.window > 0)
        see = see && (long long)t > (long long)i - a.f.window;
    return (see || j < u.prefix) && i >= 0;
}

// The score of accumulator value s in units of log2, less `base`.  f: the token's
// and the column's factor.  FORM: there may be a cap or a bias (slope, distance).
template <bool FORM>
__device__ __forceinline__ float score(const AttendArgs &a, float s, float f, float base, float slope, float distance)
{
    if (!FORM)
        return fmaf(s, f, -base);
    float x = s * f;
    if (a.f.softcap > 0.0f)  // cap tanh(y) = cap (1 - 2 / (1 + exp(2 y))); the quotient is 0 from 2^126 on
        x = (1.0f - __fdividef(2.0f, 1.0f + exp2_fast(x * (2.0f * kLog2e)))) * (a.f.softcap * kLog2e);
    if (a.f.slopes)
        x = fmaf(-slope, fabsf(distance), x);
    return x - base;
}

struct StageInfo {
    int pos[kTile];
    float k_scale[8], v_scale[8];
    int page[8];
    uint32_t came;
    uint32_t pad[3];
};

// Brings one tile's blocks into shared memory; a warp calls it.  info: which blocks came.
template <int D, bool VALUES>
__device__ __forceinline__ void load_tile(const AttendArgs &a, const CUtensorMap *kmap, const CUtensorMap *vmap, int h, int page,
                                          bool here, StageInfo &st, uint8_t *k, uint8_t *v, uint64_t *full, int lane)
{
    const int P = a.c.block;
    const uint32_t came = __ballot_sync(0xffffffffu, here && page >= 0);
    const bool pos = a.f.slopes && a.c.positions;
    if (lane == 0) {
        st.came = came;  // bit k: block k of the tile came
        mbar_expect(full, (uint32_t)__popc(came) * (uint32_t)(P * D * (VALUES ? 2 : 1) + (pos ? P * 4 : 0)));
    }
    __syncwarp();
    if (lane < 8)
        st.page[lane] = page;
    if (here && page >= 0) {
        const size_t at = (size_t)page * a.c.kv_heads + h;
        tma_load(kmap, k + lane * P * D, full, 0, 0, h, page);
        if (VALUES)
            tma_load(vmap, v + lane * P * D, full, 0, 0, h, page);
        if (pos)
            bulk_load(a.c.positions + at * P, st.pos + lane * P, (uint32_t)P * 4, full);
        copy4(a.c.k_scale + at, st.k_scale + lane);
        if (VALUES)
            copy4(a.c.v_scale + at, st.v_scale + lane);
    }
    copies_arrive(full);
}

// The segments of a CTA's stretch: units, or parts of them, in order.
template <int NT> struct Walk {
    const AttendArgs &a;
    long long at, end;
    int b, h, rt, x0, x1, count;  // tiles [x0, x1) of the unit's max(count, 1)
    Unit u;
    bool started = false;
    __device__ __forceinline__ Walk(const AttendArgs &args, const Range &r) : a(args), at(r.begin), end(r.end), b(r.b)
    {
        h = rt = x0 = x1 = count = 0;
        if (at >= end)
            return;
        // the unit that holds the first tile
        long long skip = r.skip, each = 0;
        for (int k = 0; k < a.row_tiles; ++k)
            each += max(row_unit<NT>(a, b, k).count, 1);
        h = (int)(skip / each);
        skip -= (long long)h * each;
        while (true) {
            u = row_unit<NT>(a, b, rt);
            if (skip < max(u.count, 1))
                break;
            skip -= max(u.count, 1);
            ++rt;
        }
        x0 = (int)skip;
    }
    __device__ __forceinline__ bool next()
    {
        if (started) {
            at += x1 - x0;
            if (at >= end)
                return false;
            x0 = 0;
            if (++rt == a.row_tiles) {
                rt = 0;
                if (++h == a.c.kv_heads) {
                    h = 0;
                    ++b;
                }
            }
            u = row_unit<NT>(a, b, rt);
        } else if (at >= end) {
            return false;
        }
        started = true;
        count = u.count;
        x1 = (int)min((long long)max(count, 1), x0 + (end - at));
        return true;
    }
    __device__ __forceinline__ bool whole() const { return x0 == 0 && x1 == max(count, 1); }
};

// ===========================================================================
// Attention
// ===========================================================================
// One persistent CTA per SM, 14 warps, each with one job:
//   warp 12      producer: block table, TMA of the blocks, their scales
//   warp 13      issues the products and owns the tensor memory
//   warps 4-11   softmax: two warpgroups, each NT / 2 of the columns
//   warps 0-3    add the tiles' O^T up in registers and write the results
// Per tile g: S^T(g) into one of two buffers; softmax turns it into P^T in
// shared memory; O^T(g) = V^T P^T into one of two buffers, while S^T(g + 1) is
// computed.  O^T of a tile is read out and added in 32 bits, with a power of two
// per row and tile: the weights of a tile are scaled by that tile's own maximum
// (not a running one), so a light tail after a heavy token keeps its bits.
//
// The exponents' base: exp2(x - base) in 32 bits has room for 2^127, so the base
// of a row is set at the first tile that the row sees and moves only when a later
// score passes it by 2^64 (or 2^32 in a tile that is looked at closely): no
// running maximum has to be agreed upon before the exponentials.  What the 8-bit
// weights need is the maximum's exponent only: 16-bit halves of the
// exponentials are compared two at a time in the warp (16 shuffles for 32
// columns) and four warps meet in shared memory.
constexpr int kAttendThreads = 448;

template <int D, int NT> struct AttendShared {
    static constexpr int kStages = D == 64 ? 8 : NT == 16 ? 6 : 5;
    static constexpr int kSide = kTile * D;
    alignas(1024) uint8_t tiles[kStages][2][kSide];
    alignas(1024) uint8_t q[2][NT * D];
    alignas(1024) uint8_t p[2][2][kTile * NT];
    alignas(16) Columns<NT> col;
    alignas(16) StageInfo info[kStages];
    alignas(16) uint32_t top[8][NT];   // per tile: largest exponent (biased) of exp2(x - base) * v_scale
    alignas(16) float alpha[8][NT];    // what a moved base leaves of the sums so far
    alignas(16) float warp_total[4][NT];
    alignas(16) float last_base[NT], inverse[NT];
    int highest[NT];                   // ordered bits of the largest score
    int is_set[NT];                    // the row has a base
    int moved[8][2], unset[2];
    alignas(8) uint64_t full[kStages], empty[kStages];
    uint64_t s_full[2], s_free[2], p_ready[4], o_full[2], o_free[2], q_ready, sum_ready, sum_free, drained;
    uint32_t tmem;
    int dead;
};

__device__ __forceinline__ int ordered(float x)
{
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}

// Largest of each 16-bit half over the warp, W words; lane's word index comes back in `word`.
template <int W> __device__ __forceinline__ uint32_t warp_max_halves(uint32_t *w, int lane, int &word)
{
    word = 0;
    int o = 16;
#pragma unroll
    for (int n = W; n > 1; n >>= 1, o >>= 1) {
        const bool up = lane & o;
        word = word * 2 + up;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const uint32_t send = up ? w[i] : w[i + n / 2], keep = up ? w[i + n / 2] : w[i];
            w[i] = __vmaxu2(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    }
#pragma unroll
    for (; o > 0; o >>= 1)
        w[0] = __vmaxu2(w[0], __shfl_xor_sync(0xffffffffu, w[0], o));
    return w[0];
}

template <int D, int NT, bool FORM>
__global__ void __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap)
{
    using Shared = AttendShared<D, NT>;
    constexpr int ST = Shared::kStages;
    constexpr int CW = NT / 2;                        // columns of a softmax thread
    constexpr int OC = D == 128 ? NT : NT / 2;        // columns of an adding thread
    extern __shared__ uint8_t raw[];
    Shared &sh = *(Shared *)(raw + ((1024 - (smem_u32(raw) & 1023)) & 1023));
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    volatile int *dead = &sh.dead;

    if (tid == 0) {
        sh.dead = 0;
        for (int i = 0; i < ST; ++i) {
            mbar_init(&sh.full[i], 33);  // the expected bytes, and 32 lanes' copies of scales
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_free[i], 8);
            mbar_init(&sh.o_full[i], 1);
            mbar_init(&sh.o_free[i], 4);
        }
        // four slots: tile g + 4's phase cannot complete before the adding warps have passed tile g's
        for (int i = 0; i < 4; ++i)
            mbar_init(&sh.p_ready[i], 8);
        mbar_init(&sh.drained, 1);
        mbar_init(&sh.q_ready, 8);
        mbar_init(&sh.sum_ready, 8);
        mbar_init(&sh.sum_free, 4);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < 8 * NT; i += kAttendThreads)
        ((uint32_t *)sh.top)[i] = 0;
    for (int i = tid; i < NT; i += kAttendThreads)
        sh.highest[i] = INT_MIN;
    for (int i = tid; i < ST * 8; i += kAttendThreads)
        sh.info[i >> 3].k_scale[i & 7] = sh.info[i >> 3].v_scale[i & 7] = 1.0f;
    if (wid == 13) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "r"(4 * NT)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_before();
    }
    const Range range = find_range<kAttendThreads>(a, [&](int b) {
        long long each = 0;
        for (int k = 0; k < a.row_tiles; ++k)
            each += max(row_unit<NT>(a, b, k).count, 1);
        if (blockIdx.x == 0 && !sequence(a.c, a.lengths, a.f.num_new, a.n, b, true).ok)
            report(a.status, SPEC_STATUS_BAD_LENGTH);
        return each * a.c.kv_heads;
    });
    __syncthreads();
    tc_after();
    const uint32_t tmem = sh.tmem;  // columns: S^T at 0 and NT, O^T at 2 NT and 3 NT
    const int P = a.c.block, blocks = kTile / P, log_p = 31 - __clz(P);
    Walk<NT> walk(a, range);
    if (tid == 0)
        a.joins[blockIdx.x] = make_int4(-1, 0, 0, 0);

    if (wid == 12) {
        // ---------------- producer ----------------
        if (lane < 2)
            asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &vmap : &kmap));
        int st = 0;
        uint32_t phase = 1, issued = 0;
        while (walk.next()) {
            const Unit &u = walk.u;
            if (u.count == 0)
                continue;
            const auto page_at = [&](int x) {
                const int blk = u.tile(x) * blocks + lane;
                return lane < blocks && (long long)blk * P < u.len ? a.c.block_table[(size_t)walk.b * a.c.table_stride + blk]
                                                                   : -2;
            };
            int page = page_at(walk.x0);
            for (int x = walk.x0; x < walk.x1; ++x) {
                const int next = x + 1 < walk.x1 ? page_at(x + 1) : -2;
                mbar_wait(&sh.empty[st], phase, dead);
                const bool ok = (unsigned)page < (unsigned)a.c.num_pages;
                if (page != -2 && !ok)
                    report(a.status, SPEC_STATUS_BAD_PAGE);
                if (!__any_sync(0xffffffffu, *dead)) {
                    load_tile<D, true>(a, &kmap, &vmap, walk.h, page, ok, sh.info[st], sh.tiles[st][0], sh.tiles[st][1],
                                       &sh.full[st], lane);
                    ++issued;
                }
                page = next;
                if (++st == ST) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        drain<ST>(sh.full, issued, dead, a.status);
    } else if (wid == 13) {
        // ---------------- products ----------------
        const uint32_t s_desc = instr_desc(NT, a.c.code, false, false), o_desc = instr_desc(NT, a.c.code, true, true);
        const uint64_t swizzle = D == 128 ? 2 : 4;
        int st = 0, st_prev = 0;
        uint32_t phase = 0, g = 0, seg = 0;
        bool pending = false;  // O^T of tile g - 1 is still to be issued
        const auto values = [&]() {
            const uint32_t i = (g - 1) & 1, par = ((g - 1) >> 1) & 1;
            mbar_wait(&sh.p_ready[(g - 1) & 3], ((g - 1) >> 2) & 1, dead);
            mbar_wait(&sh.o_free[i], par ^ 1, dead);
            tc_after();
            if (lane == 0) {
                const uint32_t v = smem_u32(sh.tiles[st_prev][1]), p = smem_u32(sh.p[i][0]);
#pragma unroll
                for (int k = 0; k < kTile / 32; ++k) {
                    const uint64_t vd = smem_desc(v + k * 32 * D, 0, 8 * D, swizzle);
#pragma unroll
                    for (int term = 0; term < 2; ++term)
                        tc_mma(tmem + (2 + i) * NT, vd, smem_desc(p + term * kTile * NT + k * 512, 128, kTile * 16, 0), o_desc,
                               k + term > 0);
                }
                tc_commit(&sh.o_full[i]);
                tc_commit(&sh.empty[st_prev]);
            }
            __syncwarp();
            pending = false;
        };
        while (walk.next()) {
            if (walk.u.count == 0)
                continue;
            if (pending)
                values();
            mbar_wait(&sh.q_ready, seg++ & 1, dead);
            for (int x = walk.x0; x < walk.x1; ++x) {
                const uint32_t i = g & 1, par = (g >> 1) & 1;
                mbar_wait(&sh.full[st], phase, dead);
                mbar_wait(&sh.s_free[i], par ^ 1, dead);
                tc_after();
                if (lane == 0) {
                    const uint32_t k = smem_u32(sh.tiles[st][0]), q = smem_u32(sh.q[0]);
#pragma unroll
                    for (int d = 0; d < D / 32; ++d) {
                        const uint64_t kd = smem_desc(k + d * 32, 16, 8 * D, swizzle);
#pragma unroll
                        for (int term = 0; term < 2; ++term)
                            tc_mma(tmem + i * NT, kd, smem_desc(q + term * NT * D + d * 32, 16, 8 * D, swizzle), s_desc,
                                   d + term > 0);
                    }
                    tc_commit(&sh.s_full[i]);
                }
                __syncwarp();
                if (pending)
                    values();
                ++g;
                pending = true;
                st_prev = st;
                if (++st == ST) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        if (pending)
            values();
        drain_products(&sh.drained, dead);
    } else if (wid >= 4) {
        // ---------------- softmax ----------------
        const int w = (wid - 4) >> 2, t = (tid - 128) & 127, all = tid - 128, c0 = w * CW;
        const uint32_t lanes = (uint32_t)(wid & 3) << 21;
        int st = 0;
        uint32_t phase = 0, g = 0, seg = 0;
        float l[CW], e[CW];
        while (walk.next()) {
            const Unit u = walk.u;
            if (u.count == 0)
                continue;
            named_barrier<256>(3);  // the last segment's columns are done with
            const bool tree = a.f.parent && (long long)(u.tile(walk.x1 - 1) + 1) * kTile > u.first;
            load_queries<D, NT>(a, u, walk.b, walk.h, walk.rt, tree, sh.q[0], sh.col, all);
            if (t < CW) {
                sh.col.base[c0 + t] = 0.0f;
                sh.is_set[c0 + t] = 0;
            }
            if (t == 0)
                sh.unset[w] = 1;
            proxy_fence();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.q_ready);
            named_barrier<256>(3);
            if (tree) {
                mark_kin<NT>(u, sh.col, all);
                named_barrier<256>(3);
            }
#pragma unroll
            for (int c = 0; c < CW; ++c)
                l[c] = 0.0f;
            for (int x = walk.x0; x < walk.x1; ++x) {
                const uint32_t i = g & 1, par = (g >> 1) & 1, slot = g & 7;
                mbar_wait(&sh.full[st], phase, dead);
                const StageInfo &info = sh.info[st];
                const int j0 = u.tile(x) * kTile, j = j0 + t;
                const uint32_t came = info.came;
                const bool edge = came != (1u << blocks) - 1 || !interior(a, u, j0);
                const bool cached = !edge || (j < u.len && ((came >> (t >> log_p)) & 1));
                float ks = cached ? info.k_scale[t >> log_p] : 0.0f, vs = cached ? info.v_scale[t >> log_p] : 1.0f;
                const float pos = FORM && a.f.slopes ? (a.c.positions ? (float)info.pos[t] : (float)j) : 0.0f;
                float small = info.v_scale[0];
                for (int k = 1; k < blocks; ++k)
                    small = fminf(small, info.v_scale[k]);
                bool closely = sh.unset[w] != 0 && (edge || x == walk.x0);
                closely = closely || small < 0x1p-40f;
                if (edge) {
                    // what V holds where nothing is cached, and NaN where some row sees it and some do not: neither
                    // may reach the product.  Both warpgroups look, then the first one cleans.
                    uint32_t *row = (uint32_t *)(sh.tiles[st][1] + t * D);
                    const uint32_t add = a.c.code == SPEC_E4M3 ? 0x01010101u : 0x04040404u;
                    uint32_t bad = 0;
                    for (int k = 0; k < D / 4; ++k)
                        bad |= ((row[(k + t) & (D / 4 - 1)] & 0x7f7f7f7fu) + add) & 0x80808080u;
                    named_barrier<256>(3);
                    if (w == 0 && (bad || !cached))
                        for (int k = 0; k < D / 4; ++k) {
                            const uint32_t v = row[k], nan = ((v & 0x7f7f7f7fu) + add) & 0x80808080u;
                            row[k] = cached ? v & ~((nan >> 7) * 0xffu) : 0u;
                        }
                    if (cached && bad)
                        vs = __int_as_float(0x7fffffff);
                }
                const uint32_t s_at = tmem + lanes + i * NT + c0;
                mbar_wait(&sh.s_full[i], par, dead);
                tc_after();

                // one column's score, less base
                const auto score_of = [&](int c, float s, float f, float base) {
                    return score<FORM>(a, s, ks * f, base, FORM && a.f.slopes ? sh.col.slope[c0 + c] : 0.0f,
                                       FORM && a.f.slopes ? sh.col.pos[c0 + c] - pos : 0.0f);
                };
                const auto rebase = [&]() {
                    TmemLoad<CW>::go(s_at, e);
                    tmem_wait<CW>(e);
#pragma unroll
                    for (int c = 0; c < CW; ++c) {
                        float y = score_of(c, e[c], sh.col.factor[c0 + c], 0.0f);
                        if (edge && !(cached && sees<NT>(a, u, sh.col, c0 + c, j)))
                            y = -INFINITY;
                        const int top = __reduce_max_sync(0xffffffffu, y == y ? ordered(y) : INT_MIN);
                        if (lane == 0)
                            atomicMax(&sh.highest[c0 + c], top);
                    }
                    named_barrier<128>(1 + w);
                    if (t < 32) {
                        float alpha = 1.0f;
                        bool set = true;
                        if (t < CW) {
                            const int top = sh.highest[c0 + t];
                            const float high = __int_as_float(top ^ ((top >> 31) & 0x7fffffff)), old = sh.col.base[c0 + t];
                            sh.highest[c0 + t] = INT_MIN;
                            set = sh.is_set[c0 + t];
                            if (top != INT_MIN && high > -INFINITY) {
                                if (!set || high - old > 32.0f) {
                                    const float now = ceilf(high);
                                    alpha = set ? exp2f(old - now) : 1.0f;
                                    sh.col.base[c0 + t] = now;
                                }
                                sh.is_set[c0 + t] = 1;
                                set = true;
                            }
                            set = set || sh.col.query[c0 + t] < 0;
                            sh.alpha[g & 7][c0 + t] = alpha;
                        }
                        const bool any = __any_sync(0xffffffffu, alpha != 1.0f), open = __any_sync(0xffffffffu, !set);
                        if (t == 0) {
                            sh.moved[g & 7][w] = any;
                            sh.unset[w] = open;
                        }
                    }
                    named_barrier<128>(1 + w);
                    if (sh.moved[g & 7][w]) {
#pragma unroll
                        for (int c = 0; c < CW; ++c)
                            l[c] *= sh.alpha[g & 7][c0 + c];
                    }
                };
                // exponentials into e, and the tile's largest exponents into top[slot]
                const auto exponentials = [&]() {
                    TmemLoad<CW>::go(s_at, e);
                    tmem_wait<CW>(e);
                    uint32_t half[CW / 2];
#pragma unroll
                    for (int c4 = 0; c4 < CW / 4; ++c4) {
                        const float4 f4 = ((const float4 *)(sh.col.factor + c0))[c4], b4 = ((const float4 *)(sh.col.base + c0))[c4];
                        const float f[4] = {f4.x, f4.y, f4.z, f4.w}, bs[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int c = c4 * 4 + k;
                            e[c] = exp2_fast(score_of(c, e[c], f[k], bs[k]));
                        }
                    }
                    if (edge) {
#pragma unroll
                        for (int c = 0; c < CW; ++c)
                            if (!(cached && sees<NT>(a, u, sh.col, c0 + c, j)))
                                e[c] = 0.0f;
                    }
#pragma unroll
                    for (int c = 0; c < CW; c += 2) {
                        float y0 = e[c] * vs, y1 = e[c + 1] * vs;
                        if (edge) {
                            y0 = e[c] == 0.0f ? 0.0f : y0;
                            y1 = e[c + 1] == 0.0f ? 0.0f : y1;
                        }
                        half[c / 2] = __byte_perm(__float_as_uint(y0), __float_as_uint(y1), 0x7632);
                    }
                    int word;
                    const uint32_t top = warp_max_halves<CW / 2>(half, lane, word);
                    constexpr int kSame = 32 / (CW / 2);  // lanes with the same word
                    if ((lane & (kSame - 1)) < 2) {
                        const int up = lane & 1;  // kSame >= 2: one lane for each half
                        atomicMax(&sh.top[slot][c0 + 2 * word + up], ((up ? top >> 16 : top) & 0x7fffu) >> 7);
                    }
                };
                if (t < CW)
                    sh.top[(slot + 1) & 7][c0 + t] = 0;
                if (t == 0)
                    sh.moved[g & 7][w] = 0;
                const uint4 *top4 = (const uint4 *)(sh.top[slot] + c0);
                while (true) {
                    if (closely)
                        rebase();
                    exponentials();
                    named_barrier<128>(1 + w);
                    if (closely)
                        break;
                    uint32_t most = 0;
#pragma unroll
                    for (int c4 = 0; c4 < CW / 4; ++c4) {
                        const uint4 y = top4[c4];
                        most = max(max(most, max(y.x, y.y)), max(y.z, y.w));
                    }
                    if (most < 127 + 64)
                        break;
                    // a score passed its base by 2^64 (the same verdict in the whole warpgroup): once more, closely
                    named_barrier<128>(1 + w);
                    if (t < CW)
                        sh.top[slot][c0 + t] = 0;
                    closely = true;
                }
                tc_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.s_free[i]);
                mbar_wait(&sh.o_full[i], par ^ 1, dead);  // the products of tile g - 2 have read this buffer
                uint32_t hi[CW / 4], lo[CW / 4];
#pragma unroll
                for (int c4 = 0; c4 < CW / 4; ++c4) {
                    const uint4 y = top4[c4];
                    const uint32_t ex[4] = {y.x, y.y, y.z, y.w};
                    float p[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = c4 * 4 + k;
                        // 2^(7 - exponent): the tile's largest weight of the row lands in [128, 256)
                        const float scale = __uint_as_float((261u - max(ex[k], 8u)) << 23) * vs;
                        l[c] += e[c];
                        p[k] = e[c] * scale;
                        if (edge && e[c] == 0.0f)
                            p[k] = 0.0f;
                    }
                    uint32_t first[2], rest[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t h2, back;
                        uint16_t b1, b2;
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h2) : "f"(p[2 * k + 1]), "f"(p[2 * k]));
                        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b1) : "r"(h2));
                        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(b1));
                        asm("sub.f16x2 %0, %1, %2;" : "=r"(back) : "r"(h2), "r"(back));
                        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b2) : "r"(back));
                        first[k] = b1;
                        rest[k] = b2;
                    }
                    hi[c4] = first[0] | first[1] << 16;
                    lo[c4] = rest[0] | rest[1] << 16;
                }
#pragma unroll
                for (int term = 0; term < 2; ++term) {
                    const uint32_t *b = term ? lo : hi;
                    uint8_t *dst = sh.p[i][term] + (c0 >> 4) * (kTile * 16) + t * 16 + (c0 & 15);
                    if (CW >= 16) {
#pragma unroll
                        for (int k = 0; k < CW / 16; ++k)
                            *(uint4 *)(dst + k * kTile * 16) = make_uint4(b[4 * k], b[4 * k + 1], b[4 * k + 2], b[4 * k + 3]);
                    } else {
                        *(uint2 *)dst = make_uint2(b[0], b[1]);
                    }
                }
                proxy_fence();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.p_ready[g & 3]);
                ++g;
                if (++st == ST) {
                    st = 0;
                    phase ^= 1;
                }
            }
            // the rows' totals: lanes, then four warps in shared memory
            mbar_wait(&sh.sum_free, (seg & 1) ^ 1, dead);
#pragma unroll
            for (int c = 0; c < CW; ++c) {
                float y = l[c];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    y += __shfl_xor_sync(0xffffffffu, y, o);
                if (lane == 0)
                    sh.warp_total[wid & 3][c0 + c] = y;
            }
            if (t < CW)
                sh.last_base[c0 + t] = sh.col.base[c0 + t];
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.sum_ready);
            ++seg;
        }
    } else {
        // ---------------- adding up ----------------
        const int o0 = D == 128 ? 0 : (wid >> 1) * OC, d = D == 128 ? tid : tid & 63;
        const uint32_t lanes = (uint32_t)wid << 21;
        constexpr int kPart = OC < 16 ? OC : 16;
        uint32_t g = 0, seg = 0;
        float o[OC];
        while (walk.next()) {
#pragma unroll
            for (int c = 0; c < OC; ++c)
                o[c] = 0.0f;
            const bool none = walk.u.count == 0;
            for (int x = walk.x0; x < walk.x1 && !none; ++x) {
                const uint32_t i = g & 1, par = (g >> 1) & 1;
                mbar_wait(&sh.p_ready[g & 3], (g >> 2) & 1, dead);  // top, alpha and moved of the tile
#pragma unroll
                for (int w = 0; w < 2; ++w)
                    if (sh.moved[g & 7][w]) {
#pragma unroll
                        for (int c = 0; c < OC; ++c)
                            if ((o0 + c) / CW == w)
                                o[c] *= sh.alpha[g & 7][o0 + c];
                    }
                mbar_wait(&sh.o_full[i], par, dead);
                tc_after();
#pragma unroll
                for (int c1 = 0; c1 < OC; c1 += kPart) {
                    float y[kPart];
                    TmemLoad<kPart>::go(tmem + lanes + (2 + i) * NT + o0 + c1, y);
                    tmem_wait<kPart>(y);
#pragma unroll
                    for (int c4 = 0; c4 < kPart / 4; ++c4) {
                        const uint4 ex = ((const uint4 *)(sh.top[g & 7] + o0 + c1))[c4];
                        const uint32_t x4[4] = {ex.x, ex.y, ex.z, ex.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            o[c1 + c4 * 4 + k] =
                                fmaf(y[c4 * 4 + k], __uint_as_float((max(x4[k], 8u) - 7u) << 23), o[c1 + c4 * 4 + k]);
                    }
                }
                tc_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.o_free[i]);
                ++g;
            }
            // whole units are finished here; parts go to the workspace for join_kernel
            const bool whole = walk.whole();
            const long long slot = 2ll * blockIdx.x + (walk.x0 == 0);
            const int rows = a.n * a.group;
            if (!none)
                mbar_wait(&sh.sum_ready, seg & 1, dead);
            named_barrier<128>(4);
            if (tid < NT) {
                const int r = walk.rt * NT + tid, i = r / a.group;
                float total = 0.0f, base = 0.0f;
                if (!none) {
                    total = (sh.warp_total[0][tid] + sh.warp_total[1][tid]) + (sh.warp_total[2][tid] + sh.warp_total[3][tid]);
                    base = sh.last_base[tid];
                }
                const bool live = !none && i <= walk.u.i1 && !(total == 0.0f);
                if (whole) {
                    sh.inverse[tid] = live ? 1.0f / total : 0.0f;
                    if (r < rows)
                        a.lse[((size_t)walk.b * a.n + i) * a.heads + walk.h * a.group + r % a.group] =
                            live ? (base + log2f(total)) * 0.6931471805599453f : -INFINITY;
                } else {
                    a.part_sum[slot * NT + tid] = make_float2(i <= walk.u.i1 ? total : 0.0f, base);
                }
            }
            if (!whole && walk.x1 == max(walk.count, 1) && tid == 0)
                a.joins[blockIdx.x] = make_int4((int)((walk.at - walk.x0) / range.each), walk.b, walk.h, walk.rt);
            named_barrier<128>(4);
            if (!none) {
                if (lane == 0)
                    mbar_arrive(&sh.sum_free);
                ++seg;
            }
#pragma unroll
            for (int c = 0; c < OC; ++c) {
                const int r = walk.rt * NT + o0 + c;
                if (!whole) {
                    a.part[(slot * NT + o0 + c) * D + d] = o[c];
                } else if (r < rows) {
                    const float inv = sh.inverse[o0 + c];
                    a.out[(((size_t)walk.b * a.n + r / a.group) * a.heads + walk.h * a.group + r % a.group) * D + d] =
                        __float2bfloat16(inv == 0.0f ? 0.0f : o[c] * inv);
                }
            }
        }
    }
    asm volatile("griddepcontrol.launch_dependents;");
    tc_before();
    __syncthreads();
    tc_after();
    if (wid == 13)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(4 * NT));
}

// ===========================================================================
// Weights
// ===========================================================================
// The same S^T tiles, read once more against the known lse: weight of a token
// += sum over the rows of exp2(x - lse).  A thread owns a token of its tile and
// adds its columns up, so a sum needs no other thread and no atomic.  Two
// warpgroups take alternate tiles.  Keys only: half of what attention reads.
constexpr int kWeighThreads = 320;

template <int D, int NT> struct WeighShared {
    static constexpr int kStages = 10;
    alignas(1024) uint8_t tiles[kStages][kTile * D];
    alignas(1024) uint8_t q[2][NT * D];
    alignas(16) Columns<NT> col;
    alignas(16) StageInfo info[kStages];
    alignas(8) uint64_t full[kStages], empty[kStages];
    uint64_t s_full[2], s_free[2], q_ready, drained;
    uint32_t tmem;
    int dead;
};

__device__ __forceinline__ bool covers(const Unit &u, int tile)
{
    return tile < u.head_tiles || (tile >= u.low && tile < u.low + u.count - u.head_tiles);
}

template <int D, int NT, bool FORM>
__global__ void __launch_bounds__(kWeighThreads, 1)
    weigh_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap kmap)
{
    using Shared = WeighShared<D, NT>;
    constexpr int ST = Shared::kStages;
    extern __shared__ uint8_t raw[];
    Shared &sh = *(Shared *)(raw + ((1024 - (smem_u32(raw) & 1023)) & 1023));
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    volatile int *dead = &sh.dead;
    if (tid == 0) {
        sh.dead = 0;
        for (int i = 0; i < ST; ++i) {
            mbar_init(&sh.full[i], 33);
            mbar_init(&sh.empty[i], 5);  // the products, and the four warps that read the scales
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_free[i], 4);
        }
        mbar_init(&sh.q_ready, 8);
        mbar_init(&sh.drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (wid == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "r"(2 * NT)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_before();
    }
    const Range range = find_range<kWeighThreads>(a, [&](int b) {
        if (blockIdx.x == 0 && !sequence(a.c, a.lengths, a.f.num_new, a.n, b, true).ok)
            report(a.status, SPEC_STATUS_BAD_LENGTH);
        return (long long)unit_for(a, b, 0, a.n - 1).count * a.c.kv_heads;
    });
    __syncthreads();
    tc_after();
    const uint32_t tmem = sh.tmem;
    const int P = a.c.block, blocks = kTile / P, log_p = 31 - __clz(P);
    int b = range.b;
    long long at = range.begin, skip = range.skip;
    int st = 0;
    uint32_t phase = 0, g = 0, seg = 0, issued = 0;
    // a stretch of tiles of one sequence and head; within it, the row tiles one after the other
    while (at < range.end) {
        const Unit all = unit_for(a, b, 0, a.n - 1);
        if (skip >= (long long)all.count * a.c.kv_heads) {
            skip = 0;
            ++b;
            continue;
        }
        const int h = (int)(skip / all.count), x0 = (int)(skip % all.count);
        const int x1 = (int)min((long long)all.count, x0 + (range.end - at));
        for (int rt = 0; rt < a.row_tiles; ++rt) {
            const Unit u = row_unit<NT>(a, b, rt);
            if (u.count == 0)
                continue;
            if (wid == 8) {
                // ---------------- producer ----------------
                for (int x = x0; x < x1; ++x) {
                    const int tile = all.tile(x), blk = tile * blocks + lane;
                    if (!covers(u, tile))
                        continue;
                    const bool some = lane < blocks && (long long)blk * P < u.len;
                    const int page = some ? a.c.block_table[(size_t)b * a.c.table_stride + blk] : -1;
                    const bool ok = (unsigned)page < (unsigned)a.c.num_pages;
                    if (some && !ok)
                        report(a.status, SPEC_STATUS_BAD_PAGE);
                    mbar_wait(&sh.empty[st], phase ^ 1, dead);
                    if (!__any_sync(0xffffffffu, *dead)) {
                        load_tile<D, false>(a, &kmap, nullptr, h, page, ok, sh.info[st], sh.tiles[st], nullptr, &sh.full[st],
                                            lane);
                        ++issued;
                    }
                    if (++st == ST) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            } else if (wid == 9) {
                // ---------------- products ----------------
                const uint32_t desc = instr_desc(NT, a.c.code, false, false);
                mbar_wait(&sh.q_ready, seg++ & 1, dead);
                for (int x = x0; x < x1; ++x) {
                    if (!covers(u, all.tile(x)))
                        continue;
                    mbar_wait(&sh.full[st], phase, dead);
                    mbar_wait(&sh.s_free[g & 1], ((g >> 1) & 1) ^ 1, dead);
                    tc_after();
                    if (lane == 0) {
                        const uint32_t k = smem_u32(sh.tiles[st]), q = smem_u32(sh.q[0]);
#pragma unroll
                        for (int d = 0; d < D / 32; ++d) {
                            const uint64_t kd = smem_desc(k + d * 32, 16, 8 * D, D == 128 ? 2 : 4);
#pragma unroll
                            for (int term = 0; term < 2; ++term)
                                tc_mma(tmem + (g & 1) * NT, kd,
                                       smem_desc(q + term * NT * D + d * 32, 16, 8 * D, D == 128 ? 2 : 4), desc, d + term > 0);
                        }
                        tc_commit(&sh.s_full[g & 1]);
                        tc_commit(&sh.empty[st]);
                    }
                    __syncwarp();
                    ++g;
                    if (++st == ST) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            } else {
                // ---------------- sums ----------------
                const int w = wid >> 2, t = tid & 127;
                named_barrier<256>(3);
                const bool tree = a.f.parent && (long long)(all.tile(x1 - 1) + 1) * kTile > u.first;
                load_queries<D, NT>(a, u, b, h, rt, tree, sh.q[0], sh.col, tid);
                if (tid < NT) {
                    const int r = rt * NT + tid, i = r / a.group;
                    const float lse =
                        i <= u.i1 ? a.lse_in[((size_t)b * a.n + i) * a.heads + h * a.group + r % a.group] : -INFINITY;
                    sh.col.base[tid] = lse == -INFINITY ? INFINITY : lse * kLog2e;
                }
                proxy_fence();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.q_ready);
                named_barrier<256>(3);
                if (tree) {
                    mark_kin<NT>(u, sh.col, tid);
                    named_barrier<256>(3);
                }
                for (int x = x0; x < x1; ++x) {
                    const int tile = all.tile(x);
                    if (!covers(u, tile))
                        continue;
                    if ((int)(g & 1) == w) {
                        mbar_wait(&sh.full[st], phase, dead);
                        const StageInfo &info = sh.info[st];
                        const int j0 = tile * kTile, j = j0 + t, page = info.page[t >> log_p];
                        const uint32_t came = info.came;
                        const bool edge = came != (1u << blocks) - 1 || !interior(a, u, j0);
                        const bool cached = !edge || (j < u.len && ((came >> (t >> log_p)) & 1));
                        const float ks = cached ? info.k_scale[t >> log_p] : 0.0f;
                        const float pos = FORM && a.f.slopes ? (a.c.positions ? (float)info.pos[t] : (float)j) : 0.0f;
                        float *weight = a.weights + ((size_t)(cached ? page : 0) * a.c.kv_heads + h) * P + (t & (P - 1));
                        const float before = cached ? *weight : 0.0f;
                        mbar_wait(&sh.s_full[g & 1], (g >> 1) & 1, dead);
                        tc_after();
                        float sum = 0.0f;
                        constexpr int kPart = NT < 32 ? NT : 32;
#pragma unroll 1
                        for (int c1 = 0; c1 < NT; c1 += kPart) {
                            float s[kPart];
                            TmemLoad<kPart>::go(tmem + ((uint32_t)(wid & 3) << 21) + (g & 1) * NT + c1, s);
                            tmem_wait<kPart>(s);
#pragma unroll
                            for (int c4 = 0; c4 < kPart / 4; ++c4) {
                                const float4 f4 = ((const float4 *)(sh.col.factor + c1))[c4],
                                             b4 = ((const float4 *)(sh.col.base + c1))[c4];
                                const float f[4] = {f4.x, f4.y, f4.z, f4.w}, bs[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const int c = c1 + c4 * 4 + k;
                                    const float e = exp2_fast(score<FORM>(a, s[c4 * 4 + k], ks * f[k], bs[k],
                                                                          FORM && a.f.slopes ? sh.col.slope[c] : 0.0f,
                                                                          FORM && a.f.slopes ? sh.col.pos[c] - pos : 0.0f));
                                    sum += !edge || (cached && sees<NT>(a, u, sh.col, c, j)) ? e : 0.0f;
                                }
                            }
                        }
                        tc_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&sh.s_free[g & 1]);
                            mbar_arrive(&sh.empty[st]);
                        }
                        if (cached)
                            *weight = before + sum;
                    }
                    ++g;
                    if (++st == ST) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
        }
        at += x1 - x0;
        skip += x1 - x0;
    }
    if (wid == 8)
        drain<ST>(sh.full, issued, dead, a.status);
    if (wid == 9)
        drain_products(&sh.drained, dead);
    tc_before();
    __syncthreads();
    tc_after();
    if (wid == 9)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * NT));
}

// Joins the parts of units that several CTAs worked on: CTA (c, y) joins rows
// [y * kJoinRows, ...) of the unit that ended in CTA c of attend_kernel.
constexpr int kJoinRows = 4;

template <int D, int NT> __global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ AttendArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x;
    const int4 join = a.joins[c];
    if (join.x < 0)
        return;
    constexpr int kAtOnce = 128 / D;  // rows
    const int d = threadIdx.x % D, rows = a.n * a.group;
    for (int k = threadIdx.x / D; k < kJoinRows; k += kAtOnce) {
        const int col = blockIdx.y * kJoinRows + k, r = join.w * NT + col;
        if (r >= rows)
            return;
        float top = -INFINITY;
        for (int p = join.x; p <= c; ++p) {
            const float2 s = a.part_sum[(2ll * p + (p == join.x)) * NT + col];
            if (!(s.x == 0.0f))
                top = fmaxf(top, s.y);
        }
        float total = 0.0f, o = 0.0f;
#pragma unroll 4
        for (int p = join.x; p <= c; ++p) {
            const long long at = (2ll * p + (p == join.x)) * NT + col;
            const float2 s = a.part_sum[at];
            const float w = s.x == 0.0f ? 0.0f : exp2f(s.y - top), y = a.part[at * D + d];
            total += s.x * w;
            o += s.x == 0.0f ? 0.0f : y * w;
        }
        const size_t row = ((size_t)join.y * a.n + r / a.group) * a.heads + join.z * a.group + r % a.group;
        const bool live = !(total == 0.0f);
        a.out[row * D + d] = __float2bfloat16(live ? o / total : 0.0f);
        if (d == 0)
            a.lse[row] = live ? (top + log2f(total)) * 0.6931471805599453f : -INFINITY;
    }
}

// The kernels of one head size, by columns per row tile (16, 32 or 64).
struct Kernels {
    const void *attend[3][2], *join[3], *weigh[3][2];  // [..][a cap or a bias]
    int attend_smem[3], weigh_smem[3];
};
const Kernels &kernels_d64();
const Kernels &kernels_d128();

template <int D, int NT> void fill(Kernels &k, int i)
{
    k.attend[i][0] = (const void *)attend_kernel<D, NT, false>;
    k.attend[i][1] = (const void *)attend_kernel<D, NT, true>;
    k.join[i] = (const void *)join_kernel<D, NT>;
    k.weigh[i][0] = (const void *)weigh_kernel<D, NT, false>;
    k.weigh[i][1] = (const void *)weigh_kernel<D, NT, true>;
    k.attend_smem[i] = (int)sizeof(AttendShared<D, NT>) + 1024;  // room to align
    k.weigh_smem[i] = (int)sizeof(WeighShared<D, NT>) + 1024;
    static_assert(sizeof(AttendShared<D, NT>) + 2048 <= 227 * 1024 && sizeof(WeighShared<D, NT>) + 2048 <= 227 * 1024,
                  "shared memory of a CTA");
}
template <int D> Kernels all_kernels()
{
    Kernels k{};
    fill<D, 16>(k, 0);
    fill<D, 32>(k, 1);
    fill<D, 64>(k, 2);
    return k;
}

}  // namespace specc

#endif
