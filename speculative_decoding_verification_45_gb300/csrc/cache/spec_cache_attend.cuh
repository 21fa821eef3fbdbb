// spec_cache_attend.cuh -- attention over the 8-bit key/value cache on the
// tensor cores, and the attention weight that each cached token received.
// include/spec_verify.h states the operations.
//
// The matrix products take the codes as they lie in memory: kind::f8f6f4
// multiplies 8-bit floats, so keys and values go from HBM through TMA into
// shared memory and from there into tcgen05.mma, with no conversion between.
// What multiplies them is split so that 8 bits lose next to nothing (products of
// e4m3 and e5m2 values may be mixed):
//   q    a bf16 value (8-bit significand), scaled by a power of two per row so
//        that the row's largest lies in [128, 256), as an e4m3 value and, of what
//        its 4 bits leave (8 units of the last bit at most, either sign: 3 bits),
//        an e5m2 value: exact down to 2^-14 of the row's largest element, off by
//        2^-21 of it at most below;
//   p    exp(x - ..) scaled per tile and row so that the largest lies in
//        [224, 448], rounded to 16 bits (2^-11), as two e4m3 values (2^-9 more, on
//        a grid of 2^-17 of the largest) and, with up to 32 rows a key head, an
//        e5m2 value of what they leave (2^-12 and 2^-21 in their place).  The
//        third term costs nothing at 16 columns (81 us for 64 sequences and a
//        window of 1,024) and 3% at 32 (196 us against 190 for 256 sequences of
//        1,000 to 2,000 tokens); at 48, where the softmax's instructions are the
//        time, it would cost 4 to 8% (209 against 192 us for four sequences of up
//        to 100,001 tokens, 345 against 334 for 1,000 queries).
// Each product is issued once per term into the same accumulator.
//
// Tokens are the M side (128 per tile), query rows the N side: a decode step
// has few rows (new tokens x query heads per key head), which would fill a
// fraction of an M = 128 tile, while N may be 16, 32 or 48.  So
//   S^T [128 tokens, NT rows] = K [128, D] Q^T        (K is K-major as stored)
//   O^T [D, NT rows]          = V^T [D, 128] P^T      (V is M-major as stored)
// and a thread of the softmax owns one token and all NT rows, 16 at a time, with
// every lane busy whatever the number of rows.
#ifndef SPEC_CACHE_ATTEND_CUH
#define SPEC_CACHE_ATTEND_CUH

#include <cuda.h>

#include <type_traits>

#include "spec_cache.cuh"

namespace specc {

struct AttendArgs {
    spec_cache c;
    spec_cache_form f;
    const int32_t *lengths;
    const __nv_bfloat16 *q;
    int64_t q_stride[3];
    int n, heads, group;   // group: query heads per key/value head
    uint32_t per_group;    // ceil(2^32 / group), 0 for a group of 1
    int row_tiles;         // ceil(n * group / NT)
    __nv_bfloat16 *out;
    float *lse;
    const float *lse_in;
    float *weights;
    uint8_t *split;        // [batch][kv heads][row tiles][2][NT * D]: the queries as split_kernel leaves them
    float *factor;         // [batch][kv heads][row tiles][NT]
    float *part;           // [2 * CTAs][NT][D] outputs of parts, then [2 * CTAs][NT] (total, base)
    float2 *part_sum;
    int4 *joins;           // [CTAs]: (first CTA or -1, sequence, head, row tile)
    int wait_limit;        // clocks
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
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity)  // does not wait
{
    uint32_t ok;
    asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok;
}
// Waits for a phase, `limit` clocks at most; whether it came.  When that runs
// out `dead` is set, and every wait of the CTA that is not over at once gives up.
// A role whose wait did not come uses nothing that the wait guards as an address
// or a count and goes to the end of the kernel; the threads of a warpgroup, which
// share barriers, agree on that by a vote.  (The softmax finishes its segment, on
// numbers that may not have come; they decide no address there.)
struct Guard {
    int dead, limit;
};
// NOW: a limit below the time that mbar_try itself waits (microseconds) counts as well.
template <bool NOW = false> __device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, volatile Guard *guard)
{
    if (NOW ? mbar_test(bar, parity) : mbar_try(bar, parity))
        return true;
    const uint32_t since = (uint32_t)clock();
    do {
        if (guard->dead | ((uint32_t)clock() - since > (uint32_t)guard->limit)) {
            guard->dead = 1;
            return false;
        }
    } while (!mbar_try(bar, parity));
    return true;
}

// After a wait ran out: what is in flight lands before the CTA's memory is given back (2^24 clocks at most).
__device__ __forceinline__ void land(uint64_t *bar, uint32_t parity)
{
    const long long since = clock64();
    while (!mbar_try(bar, parity) && clock64() - since < (1 << 24))
        ;
}
// The last copies into each of ST stages, `issued` in all.
template <int ST> __device__ __forceinline__ void land_stages(uint64_t *full, uint32_t issued)
{
    for (uint32_t i = 0; i < ST && i < issued; ++i)
        land(&full[i], ((issued - 1 - i) / ST) & 1);
}
__device__ __forceinline__ void tc_commit(uint64_t *bar);
__device__ __forceinline__ bool elected();
// The products of this warp.
__device__ __forceinline__ void land_products(uint64_t *bar)
{
    if (elected()) {
        tc_commit(bar);
        land(bar, 0);
    }
    __syncwarp();
}

__device__ __forceinline__ bool elected()  // one lane of a warp whose lanes are all here
{
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r;
}

template <int N> __device__ __forceinline__ void named_barrier(int id)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
}

// Barrier of N threads that also tells whether any of them brought `p`.
template <int N> __device__ __forceinline__ bool barrier_or(int id, bool p)
{
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.or.pred q, %2, %3, p;\nselp.u32 %0, 1, 0, q;\n}"
                 : "=r"(r)
                 : "r"((uint32_t)p), "r"(id), "n"(N)
                 : "memory");
    return r;
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
__device__ __forceinline__ void tmem_store16(uint32_t a, const float *r)
{
    const uint32_t *u = (const uint32_t *)r;
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(u[0]),
                 "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]),
                 "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(a)
                 : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
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

// Two 32-bit operations by one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 r;
    asm("{\n.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmul.rn.f32x2 z, x, y;\nmov.b64 {%0, %1}, z;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("{\n.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nadd.rn.f32x2 z, x, y;\nmov.b64 {%0, %1}, z;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("{\n.reg .b64 x, y, z, w;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmov.b64 z, {%6, %7};\nfma.rn.f32x2 w, x, y, "
        "z;\nmov.b64 {%0, %1}, w;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// Shared-memory matrix descriptor.  swizzle: 0 none, 2 128-byte, 4 64-byte.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint64_t swizzle)
{
    return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)((lbo >> 4) & 0x3fff) << 16 | (uint64_t)((sbo >> 4) & 0x3fff) << 32 |
           1ull << 46 | swizzle << 61;
}
// Instruction descriptor: float accumulator, M = 128; a_code 0 e4m3, 1 e5m2; B is e4m3, or e5m2 with kWideB.
constexpr uint32_t kWideB = 1u << 10;
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

__device__ __noinline__ inline Unit unit_for(const AttendArgs &a, int b, int i0, int i1)
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

// Row c of row tile rt: its query and, among its key head's, its query head.  Quotients of less than
// group + 64 come exact from the high half of a product.
struct RowAt {
    int i0, g0;
    __device__ __forceinline__ RowAt(const AttendArgs &a, int first) : i0(first / a.group), g0(first % a.group) {}
    __device__ __forceinline__ void of(const AttendArgs &a, int c, int &i, int &g) const
    {
        const uint32_t k = (uint32_t)(g0 + c), whole = a.per_group ? __umulhi(k, a.per_group) : k;
        i = i0 + (int)whole;
        g = (int)(k - whole * (uint32_t)a.group);
    }
};

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

// The tiles of all units in order, cut into equal stretches, one per CTA.
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
#pragma unroll 1
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
    alignas(16) float factor[NT];  // of the accumulator, times the token's scale: the score, in units of log2 (of softcap with one)
    float less[NT];    // weigh: the row's -lse, in units of log2
    float slope[NT];   // times -log2(e)
    float pos[NT];     // position, from origin on
    int origin;        // position of the first column's query: differences keep their bits however far out they lie
    int query[NT];     // its query, -1: none
    uint32_t nan_rows[2];  // columns, one bit each, that see a NaN value which others of its tile do not
    uint32_t kin[NT][kMaxNodes / 32];
    int up[kMaxNodes];
};
static_assert(sizeof(Columns<16>) % 16 == 0 && sizeof(Columns<48>) % 16 == 0, "copies arrive at 16 bytes");

// Pairs of 16-bit floats to 8 bits: what 4 bits hold of them, which is taken off; what 3 bits hold of the rest.
__device__ __forceinline__ uint32_t take4(uint32_t &h)
{
    uint16_t b;
    uint32_t back;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(h));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(b));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(h) : "r"(h), "r"(back));
    return b;
}
__device__ __forceinline__ uint32_t take3(uint32_t h)
{
    uint16_t b;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(b) : "r"(h));
    return b;
}
__device__ __forceinline__ uint32_t to_halves(float x0, float x1)
{
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x1), "f"(x0));
    return h;
}

// Queries as an e4m3 and an e5m2 term (for the weights two e4m3 terms), row tile by row tile, laid out as the products read
// them from shared memory (128- or 64-byte swizzled), and the factor of each
// row's accumulators; rows of `out` without a query are written here too.  A kernel of its own, D / 8 lanes a row: one warp of the
// attention kernel took 18,000 cycles for the 32 rows of a segment, as long as
// their attention over 2,000 tokens.
constexpr int kSplitRows = 4;  // rows a thread helps with, their loads in flight together

template <int D> __global__ void __launch_bounds__(256) split_kernel(const __grid_constant__ AttendArgs a, uint32_t nt)
{
    constexpr uint32_t kLanes = D / 8, kStep = 256 / kLanes;
    const uint32_t d = threadIdx.x % kLanes;
    const uint32_t units = (uint32_t)(a.c.batch * a.c.kv_heads);
    uint32_t tile[kSplitRows], c[kSplitRows];
    int b[kSplitRows], i[kSplitRows], H[kSplitRows], m[kSplitRows];
    uint4 w[kSplitRows];
#pragma unroll
    for (int k = 0; k < kSplitRows; ++k) {
        // the row, with row tiles filled up
        const uint32_t padded = (blockIdx.x * kSplitRows + k) * kStep + threadIdx.x / kLanes;
        tile[k] = padded / nt;
        c[k] = padded - tile[k] * nt;
        const uint32_t unit = tile[k] / (uint32_t)a.row_tiles, rt = tile[k] - unit * (uint32_t)a.row_tiles;
        const uint32_t r = rt * nt + c[k], q = r / (uint32_t)a.group;
        b[k] = (int)(unit / (uint32_t)a.c.kv_heads);
        i[k] = (int)q;
        H[k] = (int)((unit - b[k] * a.c.kv_heads) * a.group + (r - q * a.group));
        m[k] = -1;
        w[k] = make_uint4(0, 0, 0, 0);
        if (unit < units) {
            m[k] = sequence(a.c, a.lengths, a.f.num_new, a.n, b[k], true).m;
            if (i[k] < a.n)
                w[k] = __ldg((const uint4 *)(a.q + (size_t)b[k] * a.q_stride[0] + (size_t)i[k] * a.q_stride[1] +
                                             (size_t)H[k] * a.q_stride[2] + d * 8));
        }
    }
    asm volatile("griddepcontrol.launch_dependents;");
#pragma unroll
    for (int k = 0; k < kSplitRows; ++k) {
        if (i[k] >= m[k]) {
            w[k] = make_uint4(0, 0, 0, 0);
            if (m[k] >= 0 && i[k] < a.n && a.out) {  // a row without a query
                const size_t row = ((size_t)b[k] * a.n + i[k]) * a.heads + H[k];
                *(uint4 *)(a.out + row * D + d * 8) = w[k];
                if (d == 0)
                    a.lse[row] = -INFINITY;
            }
        }
        uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w}, most = 0;  // pairs of bf16
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int at = 16 * (e & 1);
            const uint32_t y = (x[e >> 1] >> at) & 0x7fffu;
            if (y >= 0x7f80u)  // infinities and NaN: NaN, and not the largest
                x[e >> 1] |= 0x7fffu << at;
            else
                most = max(most, y);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
            most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        // the row's power of two: its largest element becomes [128, 256)
        const int ex = most ? max((int)(most >> 7), 16) - 7 : 127;  // biased
        const float inv = __uint_as_float((uint32_t)(254 - ex) << 23);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
        {
            uint32_t h = to_halves(__uint_as_float(x[e] << 16) * inv, __uint_as_float(x[e] & 0xffff0000u) * inv);
            hi[e] = take4(h);
            lo[e] = a.out ? take3(h) : take4(h);
        }
        if (m[k] < 0)
            continue;
        uint8_t *to = a.split + (size_t)tile[k] * (2 * nt * D) + c[k] * D +
                      ((d * 8) ^ (D == 128 ? (c[k] & 7) << 4 : ((c[k] >> 1) & 3) << 4));
        *(uint2 *)to = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *(uint2 *)(to + nt * D) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        if (d == 0) {
            const float f = __uint_as_float((uint32_t)ex << 23) * a.f.scale;
            a.factor[(size_t)tile[k] * nt + c[k]] = a.f.softcap > 0.0f ? f / a.f.softcap : f * kLog2e;
        }
    }
}

// Bytes of a row tile's split queries and factors.
template <int D, int NT> constexpr uint32_t kQueryBytes = 2 * NT * D + 4 * NT;

// A row tile's split queries and factors into shared memory; one thread, which has announced the bytes.
template <int D, int NT>
__device__ __forceinline__ void load_queries(const AttendArgs &a, int b, int h, int rt, uint8_t *q, Columns<NT> &col, uint64_t *bar)
{
    const long long tile = ((long long)b * a.c.kv_heads + h) * a.row_tiles + rt;
    bulk_load(a.split + tile * (2 * NT * D), q, 2 * NT * D, bar);
    bulk_load(a.factor + tile * NT, col.factor, 4 * NT, bar);
}

// The position that token j has in its text, for the bias.
__device__ __forceinline__ int position_of(const AttendArgs &a, int b, int h, int j)
{
    if (!a.c.positions)
        return j;
    const int page = page_of(a.c, b, j / a.c.block);
    return page < 0 ? 0 : a.c.positions[((size_t)page * a.c.kv_heads + h) * a.c.block + j % a.c.block];
}

// p - origin, rounded once.
__device__ __forceinline__ float from_origin(int p, int origin)
{
    return (float)((long long)p - origin);
}

// The columns' other constants, by THREADS threads; ends without a barrier.
template <int NT, int THREADS, typename Unit>
__device__ __forceinline__ void describe_columns(const AttendArgs &a, const Unit &u, int b, int h, int rt, bool tree,
                                                 Columns<NT> &col, int t)
{
    const RowAt at(a, rt * NT);
    const int origin = a.f.slopes && at.i0 <= u.i1 ? position_of(a, b, h, u.first + at.i0) : 0;
    if (t == 0) {
        col.origin = origin;
        col.nan_rows[0] = col.nan_rows[1] = 0;
    }
    for (int c = t; c < NT; c += THREADS) {
        int i, g;
        at.of(a, c, i, g);
        const bool live = i <= u.i1;
        col.query[c] = live ? i : -1;
        if (a.f.slopes) {
            col.pos[c] = live ? from_origin(position_of(a, b, h, u.first + i), origin) : 0.0f;
            col.slope[c] = live ? -a.f.slopes[h * a.group + g] * kLog2e : 0.0f;
        }
    }
    if (tree && a.f.parent)
        for (int k = t; k < u.m; k += THREADS) {
            const int up = k > 0 ? a.f.parent[(size_t)b * a.n + k] : -1;
            if (k > 0 && (unsigned)up >= (unsigned)k)
                report(a.status, SPEC_STATUS_BAD_TREE);
            col.up[k] = (unsigned)up < (unsigned)k ? up : -1;
        }
}

// The ancestors of each column's query, after a barrier behind describe_columns.
template <int NT, int THREADS> __device__ __forceinline__ void mark_kin(Columns<NT> &col, int t)
{
    for (int c = t; c < NT; c += THREADS) {
        for (int w = 0; w < kMaxNodes / 32; ++w)
            col.kin[c][w] = 0;
        for (int k = col.query[c]; k >= 0; k = col.up[k])
            col.kin[c][k >> 5] |= 1u << (k & 31);
    }
}

// Scores in units of log2, less base (given negated), of 16 columns from c0 on; e:
// the accumulator values of a token with this scale and position.  FORM: there
// may be a cap or a bias.
template <bool FORM, int NT>
__device__ __forceinline__ void scores(const AttendArgs &a, const Columns<NT> &col, const float *less, int c0, float k_scale,
                                       float pos, float *e)
{
    const float4 *factor4 = (const float4 *)(col.factor + c0), *less4 = (const float4 *)(less + c0);
    float2 *e2 = (float2 *)e;
    const float2 k2 = make_float2(k_scale, k_scale);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float4 f = factor4[c], b = less4[c];
        const float2 f0 = mul2(k2, make_float2(f.x, f.y)), f1 = mul2(k2, make_float2(f.z, f.w));
        if (FORM) {
            e2[2 * c] = mul2(e2[2 * c], f0);
            e2[2 * c + 1] = mul2(e2[2 * c + 1], f1);
        } else {
            e2[2 * c] = fma2(e2[2 * c], f0, make_float2(b.x, b.y));
            e2[2 * c + 1] = fma2(e2[2 * c + 1], f1, make_float2(b.z, b.w));
        }
    }
    if (!FORM)
        return;
    if (a.f.softcap > 0.0f) {
        const float cap = a.f.softcap * kLog2e;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            // tanh(y) = 1 - 2 / (1 + exp(2 y)) (the quotient is 0 from 2^126 on), which cancels near 0: there the first
            // terms of its series, whose remainder is below 2^-24 of it up to 1/4
            const float y = e[c], z = y * y;
            const float series = y * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 62.0f / 2835, -17.0f / 315), 2.0f / 15), -1.0f / 3), 1.0f);
            const float whole = 1.0f - __fdividef(2.0f, 1.0f + exp2_fast(y * (2.0f * kLog2e)));
            e[c] = (fabsf(y) < 0.25f ? series : whole) * cap;
        }
    }
    if (a.f.slopes) {
        const float4 *slope4 = (const float4 *)(col.slope + c0), *from4 = (const float4 *)(col.pos + c0);  // slopes negated
        const float2 p2 = make_float2(-pos, -pos);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float4 sl = slope4[c], from = from4[c];
            float2 d0 = add2(make_float2(from.x, from.y), p2), d1 = add2(make_float2(from.z, from.w), p2);
            d0 = make_float2(fabsf(d0.x), fabsf(d0.y));
            d1 = make_float2(fabsf(d1.x), fabsf(d1.y));
            e2[2 * c] = fma2(make_float2(sl.x, sl.y), d0, e2[2 * c]);
            e2[2 * c + 1] = fma2(make_float2(sl.z, sl.w), d1, e2[2 * c + 1]);
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float4 b = less4[c];
        e2[2 * c] = add2(e2[2 * c], make_float2(b.x, b.y));
        e2[2 * c + 1] = add2(e2[2 * c + 1], make_float2(b.z, b.w));
    }
}

struct StageInfo {
    int pos[kTile];
    float k_scale[8], v_scale[8];
    int page[8];
    uint32_t came;
    uint32_t pad[3];
};

// Brings one tile's blocks of keys into shared memory, and what belongs to them; a
// warp calls it, a lane per block.
template <int D>
__device__ __forceinline__ void load_keys(const AttendArgs &a, const CUtensorMap *kmap, int h, int page, bool here, int blocks,
                                          StageInfo &st, uint8_t *k, uint64_t *full, int lane)
{
    const int P = a.c.block;
    const uint32_t came = __ballot_sync(0xffffffffu, here);
    const bool pos = a.f.slopes && a.c.positions;
    if (lane == 0) {
        st.came = came;  // bit k: block k of the tile came
        mbar_expect(full, (uint32_t)__popc(came) * (uint32_t)(P * D + (pos ? P * 4 : 0)));
    }
    __syncwarp();
    if (lane < blocks) {
        st.page[lane] = page;
        if (here) {
            const size_t at = (size_t)page * a.c.kv_heads + h;
            tma_load(kmap, k + lane * P * D, full, 0, 0, h, page);
            if (pos)
                bulk_load(a.c.positions + at * P, st.pos + lane * P, (uint32_t)P * 4, full);
            copy4(a.c.k_scale + at, st.k_scale + lane);
        }
        copies_arrive(full);
    }
}

// The segments of a CTA's stretch: units, or parts of them, in order; units
// without a tile are passed over.  A whole warp walks.
template <int NT> struct Walk {
    long long at, end;
    int b, h, rt, x0, x1;  // tiles [x0, x1) of the unit
    Unit u;
    __device__ __noinline__ void start(const AttendArgs &a, const Range &r)
    {
        at = r.begin;
        end = r.end;
        b = r.b;
        h = rt = x0 = x1 = 0;
        if (at >= end)
            return;
        // the unit that holds the first tile
        long long skip = r.skip, each = 0;
        for (int k = 0; k < a.row_tiles; ++k)
            each += row_unit<NT>(a, b, k).count;
        h = (int)(skip / max(each, 1ll));
        skip -= (long long)h * each;
        for (; rt < a.row_tiles; ++rt) {
            u = row_unit<NT>(a, b, rt);
            if (skip < u.count)
                break;
            skip -= u.count;
        }
        if (rt == a.row_tiles || h >= a.c.kv_heads) {  // lengths that changed while they were read
            at = end;
            return;
        }
        x0 = (int)skip;
        x1 = (int)min((long long)u.count, x0 + (end - at));
    }
    __device__ __noinline__ void next(const AttendArgs &a)
    {
        at += x1 - x0;
        if (at >= end)
            return;
        if (++rt == a.row_tiles || rt * NT / a.group >= u.m) {
            rt = 0;
            if (++h == a.c.kv_heads) {
                h = 0;
                // the next sequence with a query: there is one, since tiles are left
                uint32_t some;
                int b0 = b + 1 - 32;
                do {
                    b0 += 32;
                    const int k = b0 + (int)(threadIdx.x & 31);
                    some = __ballot_sync(0xffffffffu,
                                         k < a.c.batch && sequence(a.c, a.lengths, a.f.num_new, a.n, k, true).m > 0);
                } while (!some && b0 + 32 < a.c.batch);
                if (!some) {
                    at = end;
                    return;
                }
                b = b0 + __ffs(some) - 1;
            }
        }
        u = row_unit<NT>(a, b, rt);
        x0 = 0;
        x1 = (int)min((long long)u.count, end - at);
    }
};

// ===========================================================================
// Attention
// ===========================================================================
// One persistent CTA per SM, each warp with one job:
//   queries      walks the CTA's segments: describes them two ahead, brings in their split queries
//   producer     block table, TMA of the blocks, their scales (at 16 columns one
//                for keys and one for values: about 600 cycles a tile and side)
//   scores, values   issue one of the two matrix products each
//   softmax      NW warpgroups, tiles in turn; a thread owns one token and all columns
//   adding       one warpgroup: adds the tiles' O^T up in registers, writes the results
// Tile g: S^T(g) in tensor memory; warpgroup g % NW turns it into P^T in shared
// memory; O^T(g) = V^T P^T.  A tile's softmax is a chain of short dependent
// steps, so several run side by side, each on a tile of its own.
//
// O^T of a tile is read out and added in 32 bits, scaled by a power of two per
// row and tile: the weights of a tile go by that tile's own maximum (not a
// running one), so a light tail after a heavy token keeps its bits.
//
// The exponents' base: exp2(x - base) in 32 bits has room for 2^127, so a
// warpgroup keeps a row's base (0, unless the row's first scores lie far below)
// until a score passes it by 2^64, or the exponential times the value scale
// comes to 2^119: no running maximum has to be agreed upon before the
// exponentials.  What the 8-bit weights need is the maximum's exponent
// only: 16-bit halves of the exponentials are compared two at a time (9 shuffles
// for 16 columns) and the four warps meet in shared memory.
//
// What bounds it: up to 48 rows a key head, memory (2 D bytes a token; 64
// sequences of 4,000 to 8,000 tokens, 20 rows: 158 us, 5.2 TB/s; one token per
// sequence, 4 rows: 146 us, 5.6 TB/s, of 6.7 that a copy reaches), and between
// units the filling and draining of this chain, about 5,000 cycles each (256
// sequences of 1,000 to 2,000 tokens: 196 us for 828 MB).  With a cap or a bias,
// or more rows, the softmax's instructions: about 900 issue slots of an SM
// quarter for a tile of 32 columns, issued at 0.5 to 0.6 a cycle.  The program
// has to stay short: columns are taken 16 at a time by the same instructions
// (all unrolled, warps waited for instructions more than for anything else),
// exponentials and running totals live in tensor memory between the passes.
template <int D, int NT> struct AttendShape {
    static constexpr int NW = 3;                                // softmax warpgroups (four at 32 columns, with fewer registers each: 1 to 5% slower)
    static constexpr int NP = NT == 16 ? 2 : 1;                 // producers: one for each side, or one for both
    static constexpr int kThreads = 128 * (1 + NW) + 32 * (3 + NP);
    static constexpr int NO = NT == 48 ? 1 : 2;                 // O^T at a time (one: room to keep the exponentials)
    static constexpr int kBytes = kTile * D;                    // one side of a tile
    static constexpr int KS = 3, VS = D == 64 || NT == 16 ? 8 : NT >= 48 ? 5 : 6;  // tiles of keys and values in shared memory
    static constexpr int kTerms = NT <= 32 ? 3 : 2;             // of a weight (see the top)
    static constexpr int kColumns = (3 * NW + NO) * NT;         // S^T, totals and exponentials of each warpgroup, O^T
    static constexpr int kAlloc = kColumns <= 256 ? 256 : 512;
    static_assert(kColumns <= 512, "tensor memory");
    static constexpr int kRing = 8;                             // >= NW + 2 tiles between a writer and the adding warps
};

// What the other warps need to know of a segment.
struct Segment {
    int tiles;  // 0: there is none left
    int x0, head_tiles, low;
    int len, m, first, prefix, i1, b, h, rt;
    int seen_prefix, seen_low, seen_end;  // tiles that every query of the row tile sees whole: [0, ..) and [low, end)
    int whole, last;                      // the whole unit; its last part
    long long at;                         // first tile's place in the order of all
    long long rows[48];                   // of the outputs, by column; -1: none
    // k-th tile to be worked on: from the newest tokens back, since scores with a bias by distance fall that way and
    // bases set first then stay
    __device__ __forceinline__ int tile(int k) const
    {
        const int x = x0 + tiles - 1 - k;
        return x < head_tiles ? x : x - head_tiles + low;
    }
};

template <int D, int NT> struct AttendShared {
    using S = AttendShape<D, NT>;
    alignas(1024) uint8_t k[S::KS][S::kBytes];
    alignas(1024) uint8_t v[S::VS][S::kBytes];
    alignas(1024) uint8_t q[2][2][NT * D];
    alignas(1024) uint8_t p[S::NW][S::kTerms][kTile * NT];
    alignas(16) Columns<NT> col[2];
    Segment seg[4];
    alignas(16) StageInfo info[S::VS];
    alignas(16) float less[S::NW][NT];   // the exponents' bases, negated
    alignas(16) uint32_t scale[S::NW][4][NT];  // per tile: 2^k, as bits, that brings the largest weight to [224, 448]
    alignas(16) int power[S::kRing][NT];       // per tile: O^T counts 2^power, or kNothing
    alignas(16) long long out_row[NT];
    alignas(16) float factor[2][NT], inverse[NT], none[NT];  // none: bases of 0
    alignas(16) float warp_total[2][S::NW * 4][NT], last_base[2][S::NW][NT];
    alignas(16) float alpha[S::NW][NT];        // what a moved base leaves of the totals
    int highest[S::NW][NT];                    // ordered bits of the largest score
    int is_set[S::NW][NT];                     // the row has a base
    int moved[S::NW][2], unset[S::NW][2];      // by 32 columns
    alignas(8) uint64_t k_full[S::KS], k_empty[S::KS], v_full[S::VS], v_empty[S::VS];
    uint64_t s_full[S::NW], s_free[S::NW], p_ready[S::kRing], p_free[S::NW], o_full[2], o_free[2], seg_ready[4], q_ready[2];
    uint64_t sum_ready[2], sum_free[2], drained[2];
    uint32_t tmem;
    uint32_t issued[2], asked;  // copies of keys and of values, segments' queries
    Guard guard;
};

constexpr uint32_t kNoScale = 253u << 23;  // 2^126, where a tile leaves nothing to a row; others have 2^125 at most
constexpr int kNothing = INT_MIN;           // the power of such a tile's sums, and of none yet: it says nothing of the row's level

__device__ __forceinline__ int ordered(float x)
{
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}

struct MaxHalves {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return max_halves(a, b); }
};
struct MaxInt {
    __device__ __forceinline__ int operator()(int a, int b) const { return max(a, b); }
};
struct Add {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// N values per lane, combined over the warp: each lane ends with one of them, whose index comes back in `which`
// (N - 1 shuffles and what is left of the five halvings; lanes that differ only below 32 / N hold the same).
template <int N, typename T, typename Op> __device__ __forceinline__ T warp_combine(T *w, int lane, int &which, Op op)
{
    which = 0;
    int o = 16;
#pragma unroll
    for (int n = N; n > 1; n >>= 1, o >>= 1) {
        const bool up = lane & o;
        which = which * 2 + up;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const T send = up ? w[i] : w[i + n / 2], keep = up ? w[i + n / 2] : w[i];
            w[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    }
#pragma unroll
    for (; o > 0; o >>= 1)
        w[0] = op(w[0], __shfl_xor_sync(0xffffffffu, w[0], o));
    return w[0];
}

// 2^e for any e: 0 below the normal numbers, the largest power above them.
__device__ __forceinline__ float power2(int e)
{
    return e < -126 ? 0.0f : __uint_as_float((uint32_t)(min(e, 127) + 127) << 23);
}

// 2^(a - b) for a <= b + 60, the two up to 2^30 and some from 0.
__device__ __forceinline__ float power_gap(int a, int b) { return a < b - 200 ? 0.0f : power2(a - b); }

// A set of columns, one bit each.
template <int NT> using Mask = typename std::conditional<NT <= 32, uint32_t, uint64_t>::type;
template <int NT> __device__ __forceinline__ Mask<NT> low_bits(int n)
{
    return n <= 0 ? 0 : n >= NT ? ~Mask<NT>(0) >> (8 * (int)sizeof(Mask<NT>) - NT) : (Mask<NT>(1) << n) - 1;
}

// Which columns ask, and where they lie among the rows of their key head.
struct Askers {
    int first, prefix;  // of the sequence
    int i1, r0, group;  // last query, row of column 0, rows a query
};
template <int NT> __device__ __forceinline__ Mask<NT> all_columns(const Askers &k) { return low_bits<NT>((k.i1 + 1) * k.group - k.r0); }

// The columns whose queries see token j: an interval of the rows in order (row r asks from query r / group, which
// sees up to itself), or the bits of a tree.
template <int NT>
__device__ __forceinline__ Mask<NT> seen_by(const AttendArgs &a, const Askers &k, const Columns<NT> &col, int j)
{
    const Mask<NT> rows = all_columns<NT>(k);
    if (j < k.prefix)
        return rows;
    const int t = j - k.first;  // its own query, if it has one
    if (t > k.i1)
        return 0;
    Mask<NT> see = rows;
    if (t >= 0) {
        if (a.f.parent) {
            see = 0;
#pragma unroll 1
            for (int c = 0; c < NT; ++c)
                see |= Mask<NT>((col.kin[c][t >> 5] >> (t & 31)) & 1) << c;
            see &= rows;
        } else {
            see &= ~low_bits<NT>(t * k.group - k.r0);
        }
    }
    if (a.f.window > 0 && (long long)t + a.f.window <= k.i1)
        see &= low_bits<NT>(max(t + a.f.window, 0) * k.group - k.r0);  // far below, the product would pass 32 bits
    return see;
}

template <int D, int NT, bool FORM>
__global__ void __launch_bounds__((AttendShape<D, NT>::kThreads), 1)
    attend_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap)
{
    using S = AttendShape<D, NT>;
    using Shared = AttendShared<D, NT>;
    constexpr int NW = S::NW, KS = S::KS, VS = S::VS, kRing = S::kRing;
    constexpr int kQueries = 4 * (1 + NW), kScores = kQueries + 1, kValues = kQueries + 2, kProducer = kQueries + 3, NO = S::NO;
    constexpr int OC = D == 128 ? NT : NT / 2;  // columns of an adding thread
    constexpr uint32_t kO = NW * NT, kL = kO + NO * NT;  // S^T at 0, then O^T, then the totals
    extern __shared__ uint8_t raw[];
    Shared &sh = *(Shared *)(raw + ((1024 - (smem_u32(raw) & 1023)) & 1023));
    const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(0xffffffffu, tid >> 5, 0);
    volatile Guard *guard = &sh.guard;

    if (tid == 0) {
        sh.guard.dead = 0;
        sh.guard.limit = a.wait_limit;
        sh.issued[0] = sh.issued[1] = sh.asked = 0;
        for (int i = 0; i < KS; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_empty[i], 1);
        }
        for (int i = 0; i < VS; ++i) {
            mbar_init(&sh.v_full[i], 1 + kTile / a.c.block);  // the expected bytes, and each block's scales
            mbar_init(&sh.v_empty[i], 1);
        }
        for (int i = 0; i < NW; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_free[i], 4);
            mbar_init(&sh.p_free[i], 1);
        }
        for (int i = 0; i < kRing; ++i)
            mbar_init(&sh.p_ready[i], 4);
        for (int i = 0; i < 4; ++i)
            mbar_init(&sh.seg_ready[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.o_full[i], 1);
            mbar_init(&sh.o_free[i], 4);
            mbar_init(&sh.q_ready[i], 1);
            mbar_init(&sh.sum_ready[i], 4 * NW);
            mbar_init(&sh.sum_free[i], 4);
        }
        mbar_init(&sh.drained[0], 1);
        mbar_init(&sh.drained[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        a.joins[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    for (int i = tid; i < NW * 4 * NT; i += S::kThreads)
        ((uint32_t *)sh.scale)[i] = kNoScale;
    for (int i = tid; i < NW * NT; i += S::kThreads)
        ((int *)sh.highest)[i] = INT_MIN;
    for (int i = tid; i < NT; i += S::kThreads)
        sh.none[i] = 0.0f;
    if (wid == kValues) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "r"(S::kAlloc)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_before();
    }
    const Range range = find_range<S::kThreads>(a, [&](int b) {
        long long each = 0;
        for (int k = 0; k < a.row_tiles; ++k)
            each += row_unit<NT>(a, b, k).count;
        if (blockIdx.x == 0 && !sequence(a.c, a.lengths, a.f.num_new, a.n, b, true).ok)
            report(a.status, SPEC_STATUS_BAD_LENGTH);
        return each * a.c.kv_heads;
    });
    __syncthreads();
    tc_after();
    const uint32_t tmem = sh.tmem;
    const int P = a.c.block, blocks = kTile / P, log_p = 31 - __clz(P);

    if (wid == kQueries) {
        // ---------------- queries ----------------
        Walk<NT> walk;
        walk.start(a, range);
        asm volatile("griddepcontrol.wait;" ::: "memory");  // for split_kernel
        uint32_t described = 0;
        bool end = false;
#pragma unroll 1
        for (uint32_t seg = 0;; ++seg) {
            const uint32_t i = seg & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(&sh.sum_free[i], ((seg >> 1) & 1) ^ 1, guard)))
                break;  // else the segment before the last is complete
            // descriptions run two segments ahead, so that the producer need not stop between segments
            while (!end && described <= (seg ? seg + 2 : 0)) {
                const auto row_of = [&](const RowAt &at, int c) {
                    int q, g;
                    at.of(a, c, q, g);
                    return q <= walk.u.i1 ? ((long long)walk.b * a.n + q) * a.heads + walk.h * a.group + g : -1ll;
                };
                const Unit &u = walk.u;
                end = walk.at >= walk.end;
                Segment &g = sh.seg[described & 3];
                if (!end) {
                    const RowAt at(a, walk.rt * NT);
                    for (int c = lane; c < NT; c += 32)
                        g.rows[c] = row_of(at, c);
                }
                if (lane == 0) {
                    g.tiles = end ? 0 : walk.x1 - walk.x0;
                    g.x0 = walk.x0;
                    g.head_tiles = u.head_tiles;
                    g.low = u.low;
                    g.len = u.len;
                    g.m = u.m;
                    g.first = u.first;
                    g.prefix = u.prefix;
                    g.i1 = u.i1;
                    g.b = walk.b;
                    g.h = walk.h;
                    g.rt = walk.rt;
                    g.seen_prefix = u.prefix / kTile;
                    g.seen_end = (a.f.parent ? u.first : u.first + u.i0 + 1) / kTile;
                    g.seen_low = a.f.window > 0
                                     ? (int)((max((long long)u.first + u.i1 - a.f.window + 1, 0ll) + kTile - 1) / kTile)
                                     : 0;
                    g.whole = walk.x0 == 0 && walk.x1 == u.count;
                    g.last = walk.x1 == u.count;
                    g.at = walk.at;
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.seg_ready[described & 3]);
                ++described;
                if (!end)
                    walk.next(a);
            }
            const Segment &g = sh.seg[seg & 3];
            const bool some = g.tiles > 0;
            if (some) {
                const bool tree = a.f.parent && (long long)(g.tile(0) + 1) * kTile > g.first;
                describe_columns<NT, 32>(a, g, g.b, g.h, g.rt, tree, sh.col[i], lane);
                if (tree) {
                    __syncwarp();
                    mark_kin<NT, 32>(sh.col[i], lane);
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_expect(&sh.q_ready[i], some ? kQueryBytes<D, NT> : 0);
                if (some)
                    load_queries<D, NT>(a, g.b, g.h, g.rt, sh.q[i][0], sh.col[i], &sh.q_ready[i]);
            }
            if (lane == 0)
                sh.asked = seg + 1;
            if (!some)
                break;
        }
    } else if (wid >= kProducer) {
        // ---------------- producer ----------------
        const bool keys = S::NP == 1 || wid == kProducer, values = S::NP == 1 || wid != kProducer;
        if (lane < 2)
            asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &vmap : &kmap));
        int ks = 0, vs = 0;
        uint32_t k_phase = 1, v_phase = 1, k_issued = 0, v_issued = 0;
        const bool pos = a.f.slopes && a.c.positions;
        bool go = true;
        for (uint32_t seg = 0; go; ++seg) {
            if (!__all_sync(0xffffffffu, mbar_wait(&sh.seg_ready[seg & 3], (seg >> 2) & 1, guard)))
                break;
            const Segment &u = sh.seg[seg & 3];
            const int tiles = u.tiles, h = u.h;
            if (tiles == 0)
                break;
            const int32_t *table = a.c.block_table + (size_t)u.b * a.c.table_stride;
            // the table's entries 32 at a time, the next 32 on their way: a tile's entries asked for one tile ahead came
            // later than the tile was due
            const int batch = 32 / blocks;  // tiles
            const auto pages_from = [&](int x) {
                const int k = x + lane / blocks;
                if (k >= tiles)
                    return -2;
                const int blk = u.tile(k) * blocks + (lane & (blocks - 1));
                return (long long)blk * P < u.len ? max(table[blk], -1) : -2;  // -2: no block here
            };
            int pages = 0, more = pages_from(0);
            for (int x = 0; x < tiles; ++x) {
                const int at_x = x & (batch - 1);
                if (at_x == 0) {
                    pages = more;
                    more = pages_from(x + batch);
                }
                const int got = __shfl_sync(0xffffffffu, pages, (at_x * blocks + lane) & 31);
                const int page = lane < blocks ? got : -2;
                const bool ok = (unsigned)page < (unsigned)a.c.num_pages;
                if (values && page != -2 && !ok)
                    report(a.status, SPEC_STATUS_BAD_PAGE);
                const uint32_t came = __ballot_sync(0xffffffffu, ok);
                const size_t at = (size_t)max(page, 0) * a.c.kv_heads + h;
                if (keys) {
                    go = __all_sync(0xffffffffu, mbar_wait(&sh.k_empty[ks], k_phase, guard));
                    if (!go)
                        break;
                    ++k_issued;
                    if (lane == 0)
                        mbar_expect(&sh.k_full[ks], (uint32_t)__popc(came) * (uint32_t)(P * D));
                    __syncwarp();
                    if (ok)
                        tma_load(&kmap, sh.k[ks] + lane * P * D, &sh.k_full[ks], 0, 0, h, page);
                }
                if (values) {
                    go = __all_sync(0xffffffffu, mbar_wait(&sh.v_empty[vs], v_phase, guard));
                    if (!go)
                        break;
                    ++v_issued;
                    StageInfo &info = sh.info[vs];
                    if (lane == 0) {
                        info.came = came;
                        mbar_expect(&sh.v_full[vs], (uint32_t)__popc(came) * (uint32_t)(P * D + (pos ? P * 4 : 0)));
                    }
                    __syncwarp();
                    if (ok) {
                        tma_load(&vmap, sh.v[vs] + lane * P * D, &sh.v_full[vs], 0, 0, h, page);
                        if (pos)
                            bulk_load(a.c.positions + at * P, info.pos + lane * P, (uint32_t)P * 4, &sh.v_full[vs]);
                        copy4(a.c.k_scale + at, info.k_scale + lane);
                        copy4(a.c.v_scale + at, info.v_scale + lane);
                    }
                    if (lane < blocks)
                        copies_arrive(&sh.v_full[vs]);
                }
                if (++ks == KS) {
                    ks = 0;
                    k_phase ^= 1;
                }
                if (++vs == VS) {
                    vs = 0;
                    v_phase ^= 1;
                }
            }
        }
        if (keys && lane == 0)
            sh.issued[0] = k_issued;
        if (values && lane == 0)
            sh.issued[1] = v_issued;
    } else if (wid == kScores) {
        // ---------------- S^T = K Q^T ----------------
        const uint32_t desc = instr_desc(NT, a.c.code, false, false);
        constexpr uint64_t swizzle = D == 128 ? 2 : 4;
        // descriptors of the first buffers; others lie a whole number of 16 bytes further
        const uint64_t k_desc = smem_desc(smem_u32(sh.k[0]), 16, 8 * D, swizzle),
                       q_desc = smem_desc(smem_u32(sh.q[0][0]), 16, 8 * D, swizzle);
        int ks = 0, w = 0;
        uint32_t k_phase = 0, s_phase = 1;
        bool go = true;
#pragma unroll 1
        for (uint32_t seg = 0; go; ++seg) {
            if (!__all_sync(0xffffffffu, mbar_wait<true>(&sh.q_ready[seg & 1], (seg >> 1) & 1, guard)))
                break;
            const int tiles = __shfl_sync(0xffffffffu, sh.seg[seg & 3].tiles, 0);
            if (tiles == 0)
                break;
            const uint64_t qd = q_desc + (seg & 1) * (2 * NT * D >> 4);
#pragma unroll 1
            for (int x = 0; x < tiles; ++x) {
                go = __all_sync(0xffffffffu, mbar_wait(&sh.k_full[ks], k_phase, guard) && mbar_wait(&sh.s_free[w], s_phase, guard));
                if (!go)
                    break;
                tc_after();
                if (elected()) {
                    const uint64_t kd = k_desc + (uint32_t)ks * (S::kBytes >> 4);
#pragma unroll
                    for (int d = 0; d < D / 32; ++d) {
                        tc_mma(tmem + w * NT, kd + (d * 32 >> 4), qd + (d * 32 >> 4), desc, d > 0);
                        tc_mma(tmem + w * NT, kd + (d * 32 >> 4), qd + ((NT * D + d * 32) >> 4), desc | kWideB, true);
                    }
                    tc_commit(&sh.s_full[w]);
                    tc_commit(&sh.k_empty[ks]);
                }
                __syncwarp();
                w = w + 1 == NW ? 0 : w + 1;
                s_phase ^= w == 0;
                ks = ks + 1 == KS ? 0 : ks + 1;
                k_phase ^= ks == 0;
            }
        }
    } else if (wid == kValues) {
        // ---------------- O^T = V^T P^T ----------------
        const uint32_t desc = instr_desc(NT, a.c.code, true, true);
        const uint64_t v_desc = smem_desc(smem_u32(sh.v[0]), 0, 8 * D, D == 128 ? 2 : 4),
                       p_desc = smem_desc(smem_u32(sh.p[0][0]), 128, kTile * 16, 0);
        int vs = 0, w = 0;
        uint32_t v_phase = 0, g = 0;
        bool go = true;
#pragma unroll 1
        for (uint32_t seg = 0; go; ++seg) {
            if (!__all_sync(0xffffffffu, mbar_wait(&sh.seg_ready[seg & 3], (seg >> 2) & 1, guard)))
                break;
            const int tiles = __shfl_sync(0xffffffffu, sh.seg[seg & 3].tiles, 0);
            if (tiles == 0)
                break;
#pragma unroll 1
            for (int x = 0; x < tiles; ++x) {
                const uint32_t i = g % NO;
                go = __all_sync(0xffffffffu, mbar_wait(&sh.p_ready[g % kRing], (g / kRing) & 1, guard) &&
                                                 mbar_wait(&sh.v_full[vs], v_phase, guard) &&
                                                 mbar_wait(&sh.o_free[i], ((g / NO) & 1) ^ 1, guard));
                if (!go)
                    break;
                tc_after();
                if (elected()) {
                    const uint64_t vd = v_desc + (uint32_t)vs * (S::kBytes >> 4),
                                   pd = p_desc + (uint32_t)w * (S::kTerms * kTile * NT >> 4);
                    const uint32_t d = tmem + kO + i * NT;
#pragma unroll
                    for (int k = 0; k < kTile / 32; ++k) {
                        tc_mma(d, vd + (k * 32 * D >> 4), pd + (k * 512 >> 4), desc, k > 0);
                        tc_mma(d, vd + (k * 32 * D >> 4), pd + ((kTile * NT + k * 512) >> 4), desc, true);
                        if (S::kTerms == 3)
                            tc_mma(d, vd + (k * 32 * D >> 4), pd + ((2 * kTile * NT + k * 512) >> 4), desc | kWideB, true);
                    }
                    tc_commit(&sh.o_full[i]);
                    tc_commit(&sh.p_free[w]);
                    tc_commit(&sh.v_empty[vs]);
                }
                __syncwarp();
                ++g;
                w = w + 1 == NW ? 0 : w + 1;
                vs = vs + 1 == VS ? 0 : vs + 1;
                v_phase ^= vs == 0;
            }
        }
    } else if (wid >= 4) {
        // ---------------- softmax ----------------
        const int w = (wid >> 2) - 1, t = tid & 127, bar = 1 + w;
        const uint32_t lanes = (uint32_t)(wid & 3) << 21, s_at = tmem + lanes + w * NT, l_at = s_at + kL, e_at = l_at + NW * NT;
        int vs = 0, turn = 0;  // turn: whose tile it is
        uint32_t v_phase = 0, g = 0, mine = 0;
#pragma unroll 1
        for (uint32_t seg = 0;; ++seg) {
            const bool came_here = mbar_wait(&sh.q_ready[seg & 1], (seg >> 1) & 1, guard);
            const Segment &u = sh.seg[seg & 3];
            Columns<NT> &col = sh.col[seg & 1];
            const int tiles = came_here ? u.tiles : 0;
            if (barrier_or<128>(bar, tiles == 0))
                break;
            bool fresh = true;  // no tile of this segment yet
            {
                const float zero[16] = {};
                for (int c0 = 0; c0 < NT; c0 += 16)
                    tmem_store16(l_at + c0, zero);
                tmem_store_wait();
            }
            if (t < NT) {
                sh.less[w][t] = 0.0f;
                sh.is_set[w][t] = 0;
            }
#pragma unroll 1
            for (int x = 0; x < tiles; ++x) {
                if (turn == w) {
                    mbar_wait(&sh.v_full[vs], v_phase, guard);
                    const StageInfo &info = sh.info[vs];
                    const int tile = u.tile(x), j = tile * kTile + t;
                    const uint32_t came = info.came;
                    float k_scale = info.k_scale[t >> log_p], v_scale = info.v_scale[t >> log_p];
                    const float pos = FORM && a.f.slopes ? from_origin(a.c.positions ? info.pos[t] : j, col.origin) : 0.0f;
                    const bool edge = came != (1u << blocks) - 1 ||
                                      !(tile < u.seen_prefix || (tile >= u.seen_low && tile < u.seen_end));
                    const bool check = fresh || sh.unset[w][0] || (NT > 32 && sh.unset[w][1]);
                    bool closely = false;
                    Mask<NT> see = ~Mask<NT>(0);
                    float v_most = v_scale;
                    if (edge) {
                        const bool cached = j < u.len && ((came >> (t >> log_p)) & 1);
                        const Askers askers{u.first, u.prefix, u.i1, u.rt * NT, a.group};
                        see = cached ? seen_by<NT>(a, askers, col, j) : 0;
                        const bool all = see == all_columns<NT>(askers);
                        v_scale = v_most = see ? v_scale : 0.0f;
                        uint4 *row = (uint4 *)(sh.v[vs] + t * D);
                        if (!cached) {  // nothing was loaded here
                            k_scale = 0.0f;
#pragma unroll 1
                            for (int k = 0; k < D / 16; ++k)
                                row[(k + t) & (D / 16 - 1)] = make_uint4(0, 0, 0, 0);
                        } else if (!all) {
                            // a NaN that some row does not see must not reach the product: 0 stands in its place, and
                            // the rows that do see it are noted
                            const uint32_t add = a.c.code == SPEC_E4M3 ? 0x01010101u : 0x04040404u;
                            uint32_t bad = 0;
#pragma unroll 4
                            for (int k = 0; k < D / 16; ++k) {
                                const uint4 v = row[(k + t) & (D / 16 - 1)];
                                bad |= ((v.x & 0x7f7f7f7fu) + add) | ((v.y & 0x7f7f7f7fu) + add) |
                                       ((v.z & 0x7f7f7f7fu) + add) | ((v.w & 0x7f7f7f7fu) + add);
                            }
                            if (bad & 0x80808080u) {
#pragma unroll 1
                                for (int k = 0; k < D / 4; ++k) {
                                    const uint32_t v = ((uint32_t *)row)[k], nan = ((v & 0x7f7f7f7fu) + add) & 0x80808080u;
                                    ((uint32_t *)row)[k] = v & ~((nan >> 7) * 0xffu);
                                }
                                atomicOr(&col.nan_rows[0], (uint32_t)see);
                                if (NT > 32)
                                    atomicOr(&col.nan_rows[1], (uint32_t)((uint64_t)see >> 32));
                            }
                        }
                        __syncwarp();
                    }
                    // the largest scale among the warp's blocks (positive: the bits order as they do)
                    v_most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v_most)));
                    uint32_t *scales = sh.scale[w][mine & 3];
                    mbar_wait(&sh.s_full[w], mine & 1, guard);
                    tc_after();

                    if (t < NT)
                        sh.scale[w][(mine + 1) & 3][t] = kNoScale;
                    const auto exponentials = [&](int c0, float *e) {
                        TmemLoad<16>::go(s_at + c0, e);
                        tmem_wait<16>(e);
                        scores<FORM>(a, col, sh.less[w], c0, k_scale, pos, e);
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            e[c] = exp2_fast(e[c]);
                        if (edge) {
                            const uint32_t bits = (uint32_t)(see >> c0);
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                e[c] = (bits >> c) & 1 ? e[c] : 0.0f;
                        }
                    };
                    while (true) {
                        if (closely) {
                            // bases from the rows' largest scores
#pragma unroll 1
                            for (int c0 = 0; c0 < NT; c0 += 16) {
                                alignas(8) float e[16];
                                TmemLoad<16>::go(s_at + c0, e);
                                tmem_wait<16>(e);
                                scores<FORM>(a, col, sh.none, c0, k_scale, pos, e);
                                int key[16], which;
                                const uint32_t bits = (uint32_t)(see >> c0);
#pragma unroll
                                for (int c = 0; c < 16; ++c)
                                    key[c] = ((bits >> c) & 1) && e[c] == e[c] ? ordered(e[c]) : INT_MIN;
                                const int most = warp_combine<16>(key, lane, which, MaxInt());
                                if ((lane & 1) == 0)
                                    atomicMax(&sh.highest[w][c0 + which], most);
                            }
                            named_barrier<128>(bar);
                            if (t < (NT + 31) / 32 * 32) {
                                float alpha = 1.0f;
                                bool set = true;
                                if (t < NT) {
                                    const int top = sh.highest[w][t];
                                    const float high = __int_as_float(top ^ ((top >> 31) & 0x7fffffff)), old = -sh.less[w][t];
                                    sh.highest[w][t] = INT_MIN;
                                    set = sh.is_set[w][t];
                                    if (top != INT_MIN && high > -INFINITY) {
                                        if (!set || high > old) {
                                            const float now = fminf(fmaxf(ceilf(high), -0x1p30f), 0x1p30f);
                                            alpha = set ? exp2f(old - now) : 1.0f;
                                            sh.less[w][t] = -now;
                                        }
                                        sh.is_set[w][t] = 1;
                                        set = true;
                                    }
                                    set = set || col.query[t] < 0;
                                    sh.alpha[w][t] = alpha;
                                }
                                const bool any = __any_sync(0xffffffffu, alpha != 1.0f), open = __any_sync(0xffffffffu, !set);
                                if (lane == 0) {
                                    sh.moved[w][t >> 5] = any;
                                    sh.unset[w][t >> 5] = open;
                                }
                            }
                            named_barrier<128>(bar);
                            if (sh.moved[w][0] || (NT > 32 && sh.moved[w][1])) {
#pragma unroll 1
                                for (int c0 = 0; c0 < NT; c0 += 16) {
                                    float y[16];
                                    TmemLoad<16>::go(l_at + c0, y);
                                    tmem_wait<16>(y);
#pragma unroll
                                    for (int c = 0; c < 16; ++c)
                                        y[c] *= sh.alpha[w][c0 + c];
                                    tmem_store16(l_at + c0, y);
                                }
                                tmem_store_wait();
                            }
                        }
                        // exponentials, and what the tile's largest weight of each row has to be scaled by
                        bool again = false;
#pragma unroll 1
                        for (int c0 = 0; c0 < NT; c0 += 16) {
                            alignas(8) float e[16];
                            exponentials(c0, e);
                            tmem_store16(e_at + c0, e);
                            uint32_t half[8];
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                half[c] = __byte_perm(__float_as_uint(e[2 * c]), __float_as_uint(e[2 * c + 1]), 0x7632);
                            int which;
                            const uint32_t two = warp_combine<8>(half, lane, which, MaxHalves());
                            const uint32_t most = lane & 1 ? two & 0xffff0000u : two << 16;  // a float, cut to 16 bits
                            // 2^k with 224 <= 2^k * largest weight <= 448 (448 = 1.75 * 2^8)
                            const uint32_t largest = __float_as_uint(__uint_as_float(most) * v_most), top = (largest + (0x1fu << 16)) >> 23;
                            again = again || most >= 191u << 23 || largest >= 246u << 23;
                            if ((lane & 3) < 2) {
                                const int c = c0 + 2 * which + (lane & 1);
                                atomicMin(&scales[c], (262u - max(top, 9u + min(top, 1u))) << 23);
                                if (check && !closely)
                                    atomicMax(&sh.highest[w][c], (int)min(most, largest));
                            }
                        }
                        // a score that passed its base by 2^64, or by what brings it to 2^119 with its scale, sends the
                        // warpgroup round again
                        bool redo = barrier_or<128>(bar, again && !closely);
                        if (check && !closely) {
                            // rows without a base keep 0 if their largest exponential, alone and times the scale, is not
                            // far below 1
                            bool low = false;
                            if (t < NT) {
                                low = !sh.is_set[w][t] && col.query[t] >= 0;
                                if (low && sh.highest[w][t] >= 67 << 23) {
                                    sh.is_set[w][t] = 1;
                                    low = false;
                                }
                                sh.highest[w][t] = INT_MIN;
                            }
                            if (t == 0)
                                sh.unset[w][0] = sh.unset[w][1] = 0;
                            redo = barrier_or<128>(bar, low) || redo;
                        }
                        if (!redo)
                            break;
                        if (t < NT)
                            scales[t] = kNoScale;
                        closely = true;
                    }
                    tmem_store_wait();
                    tc_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sh.s_free[w]);
                    if (t < NT)
                        sh.power[g % kRing][t] =
                            scales[t] == kNoScale ? kNothing : 127 - (int)(scales[t] >> 23) - (int)sh.less[w][t];
                    mbar_wait(&sh.p_free[w], (mine & 1) ^ 1, guard);
#pragma unroll 1
                    for (int c0 = 0; c0 < NT; c0 += 16) {
                        alignas(8) float e[16], l[16];
                        TmemLoad<16>::go(l_at + c0, l);
                        TmemLoad<16>::go(e_at + c0, e);
                        tmem_wait<16>(e);
                        tmem_wait<16>(l);
                        const float2 v2 = make_float2(v_scale, v_scale);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            ((float2 *)l)[c] = add2(((float2 *)l)[c], ((float2 *)e)[c]);
                        tmem_store16(l_at + c0, l);
                        uint32_t hi[4], lo[4], rest[4];
#pragma unroll
                        for (int c4 = 0; c4 < 4; ++c4) {
                            const float4 y = *(const float4 *)(scales + c0 + c4 * 4);
                            // e * v first: y * v may pass the floats where e is 0
                            const float2 p0 = mul2(mul2(((float2 *)e)[2 * c4], v2), make_float2(y.x, y.y)),
                                         p1 = mul2(mul2(((float2 *)e)[2 * c4 + 1], v2), make_float2(y.z, y.w));
                            uint32_t h0 = to_halves(p0.x, p0.y), h1 = to_halves(p1.x, p1.y);
                            hi[c4] = take4(h0) | take4(h1) << 16;
                            lo[c4] = take4(h0) | take4(h1) << 16;
                            rest[c4] = take3(h0) | take3(h1) << 16;
                        }
                        uint8_t *dst = sh.p[w][0] + (c0 >> 4) * (kTile * 16) + t * 16;
                        *(uint4 *)dst = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *(uint4 *)(dst + kTile * NT) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        if (S::kTerms == 3)
                            *(uint4 *)(dst + 2 * kTile * NT) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
                    }
                    tmem_store_wait();
                    proxy_fence();
                    tc_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sh.p_ready[g % kRing]);
                    ++mine;
                    fresh = false;
                }
                ++g;
                turn = turn + 1 == NW ? 0 : turn + 1;
                if (++vs == VS) {
                    vs = 0;
                    v_phase ^= 1;
                }
            }
            // the rows' totals, warp by warp
            if (barrier_or<128>(bar, !mbar_wait(&sh.sum_free[seg & 1], ((seg >> 1) & 1) ^ 1, guard)))
                break;
            if (t < NT)
                sh.last_base[seg & 1][w][t] = -sh.less[w][t];
#pragma unroll 1
            for (int c0 = 0; c0 < NT; c0 += 16) {
                float y[16];
                int which;
                TmemLoad<16>::go(l_at + c0, y);
                tmem_wait<16>(y);
                const float sum = warp_combine<16>(y, lane, which, Add());
                if ((lane & 1) == 0)
                    sh.warp_total[seg & 1][w * 4 + (wid & 3)][c0 + which] = sum;
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.sum_ready[seg & 1]);
        }
        tmem_store_wait();
    } else {
        // ---------------- adding up ----------------
        const int o0 = D == 128 ? 0 : (wid >> 1) * OC, d = D == 128 ? tid : tid & 63, bar = 1 + NW;
        const uint32_t lanes = (uint32_t)wid << 21;
        constexpr int kPart = OC % 16 == 0 ? 16 : 8;
        uint32_t g = 0;
        alignas(8) float o[OC];
#pragma unroll 1
        for (uint32_t seg = 0;; ++seg) {
            bool lost = !mbar_wait(&sh.seg_ready[seg & 3], (seg >> 2) & 1, guard), stop = false;
            const Segment &u = sh.seg[seg & 3];
            const int tiles = lost ? 0 : u.tiles;
            if (barrier_or<128>(bar, tiles == 0))
                break;
#pragma unroll
            for (int c = 0; c < OC; ++c)
                o[c] = 0.0f;
            int ref = kNothing;  // of column tid: its sums count 2^ref
#pragma unroll 1
            for (int x = 0; x < tiles; ++x) {
                const uint32_t i = g & 1, io = g % NO;
                lost = !mbar_wait(&sh.p_ready[g % kRing], (g / kRing) & 1, guard) || lost;  // the tile's powers
                bool moved = false;
                float alpha = 1.0f;
                if (tid < NT) {
                    const int power = sh.power[g % kRing][tid];
                    if (ref == kNothing) {
                        ref = power;
                    } else if (power > ref + 60) {
                        alpha = power_gap(ref, power);
                        ref = power;
                        moved = true;
                    }
                    sh.factor[i][tid] = power == kNothing ? 0.0f : power_gap(power, ref);
                }
                if (barrier_or<128>(bar, moved || lost)) {
                    if (tid < NT)
                        sh.inverse[tid] = alpha;
                    stop = barrier_or<128>(bar, lost);
                    if (stop)
                        break;
#pragma unroll
                    for (int c = 0; c < OC; ++c)
                        o[c] *= sh.inverse[o0 + c];
                }
                lost = !mbar_wait(&sh.o_full[io], (g / NO) & 1, guard);
                tc_after();
#pragma unroll
                for (int c1 = 0; c1 < OC; c1 += kPart) {
                    float y[kPart];
                    TmemLoad<kPart>::go(tmem + lanes + kO + io * NT + o0 + c1, y);
                    tmem_wait<kPart>(y);
#pragma unroll
                    for (int c = 0; c < kPart; c += 4) {
                        const float4 f = *(const float4 *)(sh.factor[i] + o0 + c1 + c);
                        float2 *o2 = (float2 *)(o + c1 + c);
                        o2[0] = fma2(make_float2(y[c], y[c + 1]), make_float2(f.x, f.y), o2[0]);
                        o2[1] = fma2(make_float2(y[c + 2], y[c + 3]), make_float2(f.z, f.w), o2[1]);
                    }
                }
                tc_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.o_free[io]);
                ++g;
            }
            if (stop)
                break;
            // whole units are finished here; parts go to the workspace for join_kernel
            const bool whole = u.whole;
            const long long slot = 2ll * blockIdx.x + (u.x0 == 0);
            lost = !mbar_wait(&sh.sum_ready[seg & 1], (seg >> 1) & 1, guard) || lost;
            if (barrier_or<128>(bar, lost))
                break;
            bool far = false;
            if (tid < NT) {
                float total = 0.0f, base = 0.0f, part[NW];
                if (sh.col[seg & 1].query[tid] >= 0) {
                    bool any = false;
                    const float(*y)[NT] = sh.warp_total[seg & 1], (*last)[NT] = sh.last_base[seg & 1];
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        part[w] = (y[4 * w][tid] + y[4 * w + 1][tid]) + (y[4 * w + 2][tid] + y[4 * w + 3][tid]);
                        if (!(part[w] == 0.0f)) {
                            base = any ? fmaxf(base, last[w][tid]) : last[w][tid];
                            any = true;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < NW; ++w)
                        total += part[w] == 0.0f ? 0.0f : part[w] * exp2f(last[w][tid] - base);
                }
                const bool live = !(total == 0.0f);
                const long long row = u.rows[tid];
                sh.out_row[tid] = row;
                // sums count 2^ref, totals 2^base
                int up = 0;
                const float significand = isfinite(total) ? frexpf(total, &up) : __int_as_float(0x7fffffff);
                const int level = (int)max(min((long long)ref - (long long)base - up, 250ll), -250ll);
                far = live && abs(level) > 100;  // a power that no float may hold goes in two
                const int first = far ? level / 2 : 0;
                sh.factor[0][tid] = power2(first);
                sh.inverse[tid] = live && ref != kNothing ? power2(level - first) / significand : 0.0f;
                if (sh.col[seg & 1].nan_rows[tid >> 5] >> (tid & 31) & 1) {
                    sh.inverse[tid] = __int_as_float(0x7fffffff);
                    if (!whole && !live) {  // a part of no weight has to be joined all the same
                        total = 0x1p-126f;
                        base = -0x1p30f;
                    }
                }
                if (whole) {
                    if (row >= 0)
                        a.lse[row] = live ? (base + log2f(total)) * 0.6931471805599453f : -INFINITY;
                } else {
                    a.part_sum[slot * NT + tid] = make_float2(total, base);
                }
            }
            if (!whole && u.last && tid == 0)
                a.joins[blockIdx.x] = make_int4((int)((u.at - u.x0) / range.each), u.b, u.h, u.rt);
            if (barrier_or<128>(bar, far)) {
#pragma unroll
                for (int c = 0; c < OC; ++c)
                    o[c] *= sh.factor[0][o0 + c];
            }
            if (lane == 0)  // the segment's place is free
                mbar_arrive(&sh.sum_free[seg & 1]);
            if (whole) {
#pragma unroll
                for (int c = 0; c < OC; ++c) {
                    const float inv = sh.inverse[o0 + c];
                    const long long row = sh.out_row[o0 + c];
                    if (row >= 0)
                        a.out[row * D + d] = __float2bfloat16(inv == 0.0f ? 0.0f : o[c] * inv);
                }
            } else {
                float *part = a.part + (slot * NT + o0) * D + d;
#pragma unroll
                for (int c = 0; c < OC; ++c) {
                    const float inv = sh.inverse[o0 + c];
                    part[c * D] = inv == 0.0f ? 0.0f : o[c] * inv;
                }
            }
        }
    }
    asm volatile("griddepcontrol.launch_dependents;");
    tc_before();
    __syncthreads();
    tc_after();
    if (guard->dead) {
        if (wid == kQueries) {
            for (uint32_t k = 1; k <= 2 && k <= sh.asked; ++k)
                land(&sh.q_ready[(sh.asked - k) & 1], ((sh.asked - k) >> 1) & 1);
        } else if (wid >= kProducer) {
            if (S::NP == 1 || wid == kProducer)
                land_stages<KS>(sh.k_full, sh.issued[0]);
            if (S::NP == 1 || wid != kProducer)
                land_stages<VS>(sh.v_full, sh.issued[1]);
        } else if (wid == kScores || wid == kValues) {
            land_products(&sh.drained[wid == kValues]);
        }
        if (tid == 0)
            report(a.status, SPEC_STATUS_INTERNAL);
        __syncthreads();
    }
    if (wid == kValues)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kAlloc));
}


// ===========================================================================
// Weights
// ===========================================================================
// The same S^T tiles, read once more against the known lse: weight of a token
// += sum over the rows of exp2(x - lse).  A thread owns a token of its tile and
// adds its columns up, so a sum needs no other thread and no atomic.  One product
// makes both terms of the queries, side by side; so both are e4m3 values, exact
// down to 2^-10 of the row's largest element and off by 2^-17 of it at most below
// (an e5m2 term needs a product of its own: 54 us against 52 for 32 sequences of
// 8192 tokens).  Three
// warpgroups take tiles in turn.  Keys only: half of what attention reads.
constexpr int kWeighGroups = 3;  // 32 sequences of 8192 tokens took 55 us when it was chosen (51 now); two 60, four 56
constexpr int kWeighThreads = 128 * kWeighGroups + 96;

template <int D, int NT> struct WeighShared {
    static constexpr int kStages = 10, kAlloc = 2 * NT * kWeighGroups <= 128 ? 128 : 2 * NT * kWeighGroups <= 256 ? 256 : 512;
    alignas(1024) uint8_t tiles[kStages][kTile * D];
    alignas(1024) uint8_t q[2][NT * D];
    alignas(16) Columns<NT> col;
    alignas(16) StageInfo info[kStages];
    alignas(8) uint64_t full[kStages], empty[kStages];
    uint64_t s_full[kWeighGroups], s_free[kWeighGroups], q_ready, drained;
    uint32_t tmem;
    uint32_t issued[2], asked;  // tiles up to the last one of each producer, row tiles' queries
    Guard guard;
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
    constexpr int ST = Shared::kStages, NW = kWeighGroups, kProducts = 4 * NW, kProducer = kProducts + 1;
    extern __shared__ uint8_t raw[];
    Shared &sh = *(Shared *)(raw + ((1024 - (smem_u32(raw) & 1023)) & 1023));
    const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(0xffffffffu, tid >> 5, 0);
    volatile Guard *guard = &sh.guard;
    if (tid == 0) {
        sh.guard.dead = 0;
        sh.guard.limit = a.wait_limit;
        sh.issued[0] = sh.issued[1] = sh.asked = 0;
        for (int i = 0; i < ST; ++i) {
            mbar_init(&sh.full[i], 1 + kTile / a.c.block);  // the expected bytes, and each block's scales
            mbar_init(&sh.empty[i], 5);  // the products, and the four warps that read the scales
        }
        for (int i = 0; i < kWeighGroups; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_free[i], 4);
        }
        mbar_init(&sh.q_ready, 1);
        mbar_init(&sh.drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (wid == kProducts) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "r"(Shared::kAlloc)
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
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for split_kernel
    const int P = a.c.block, blocks = kTile / P, log_p = 31 - __clz(P);
    int b = range.b;
    long long at = range.begin, skip = range.skip;
    int st = 0;
    uint32_t phase = 0, g = 0, seg = 0;
    bool go = true;
    // a stretch of tiles of one sequence and head; within it, the row tiles one after the other
    while (go && at < range.end) {
        const Unit all = unit_for(a, b, 0, a.n - 1);
        if (skip >= (long long)all.count * a.c.kv_heads) {
            skip = 0;
            if (++b == a.c.batch)
                break;
            continue;
        }
        const int h = (int)(skip / all.count), x0 = (int)(skip % all.count);
        const int x1 = (int)min((long long)all.count, x0 + (range.end - at));
        for (int rt = 0; go && rt < a.row_tiles; ++rt) {
            const Unit u = row_unit<NT>(a, b, rt);
            const int low = all.tile(x0), high = all.tile(x1 - 1);
            if (u.count == 0 || !(low < u.head_tiles || (high >= u.low && low < u.low + u.count - u.head_tiles)))
                continue;  // no tile of the stretch
            if (wid >= kProducer) {
                // ---------------- producer ----------------
                const int32_t *table = a.c.block_table + (size_t)b * a.c.table_stride;
                const int batch = 32 / blocks;  // tiles whose table entries come together, a batch ahead
                const auto pages_from = [&](int x) {
                    const int k = x + lane / blocks;
                    if (k >= x1)
                        return -2;
                    const int blk = all.tile(k) * blocks + (lane & (blocks - 1));
                    return (long long)blk * P < u.len ? max(table[blk], -1) : -2;  // -2: no block here
                };
                int pages = 0, more = pages_from(x0);
                for (int x = x0; x < x1; ++x) {
                    const int at_x = (x - x0) & (batch - 1);
                    if (at_x == 0) {
                        pages = more;
                        more = pages_from(x + batch);
                    }
                    const int got = __shfl_sync(0xffffffffu, pages, (at_x * blocks + lane) & 31);
                    if (!covers(u, all.tile(x)))
                        continue;
                    const int page = lane < blocks ? got : -2;
                    const bool ok = (unsigned)page < (unsigned)a.c.num_pages;
                    if (page != -2 && !ok)
                        report(a.status, SPEC_STATUS_BAD_PAGE);
                    if ((int)(g++ & 1) == wid - kProducer) {  // two producers, tiles in turn
                        go = __all_sync(0xffffffffu, mbar_wait(&sh.empty[st], phase ^ 1, guard));
                        if (!go)
                            break;
                        load_keys<D>(a, &kmap, h, page, ok, blocks, sh.info[st], sh.tiles[st], &sh.full[st], lane);
                        if (lane == 0)
                            sh.issued[wid - kProducer] = g;
                    }
                    if (++st == ST) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            } else if (wid == kProducts) {
                // ---------------- products ----------------
                const uint32_t desc = instr_desc(2 * NT, a.c.code, false, false);  // both terms' columns side by side
                go = __all_sync(0xffffffffu, mbar_wait<true>(&sh.q_ready, seg++ & 1, guard));
                for (int x = x0; go && x < x1; ++x) {
                    if (!covers(u, all.tile(x)))
                        continue;
                    go = __all_sync(0xffffffffu, mbar_wait(&sh.full[st], phase, guard) &&
                                                     mbar_wait(&sh.s_free[g % NW], ((g / NW) & 1) ^ 1, guard));
                    if (!go)
                        break;
                    tc_after();
                    if (elected()) {
                        const uint64_t kd = smem_desc(smem_u32(sh.tiles[st]), 16, 8 * D, D == 128 ? 2 : 4),
                                       qd = smem_desc(smem_u32(sh.q[0]), 16, 8 * D, D == 128 ? 2 : 4);
#pragma unroll
                        for (int d = 0; d < D / 32; ++d)
                            tc_mma(tmem + (g % NW) * 2 * NT, kd + (d * 32 >> 4), qd + (d * 32 >> 4), desc, d > 0);
                        tc_commit(&sh.s_full[g % NW]);
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
                const Askers askers{u.first, u.prefix, u.i1, rt * NT, a.group};
                go = !barrier_or<128 * NW>(3, guard->dead);
                if (!go)
                    break;
                const bool tree = a.f.parent && (long long)(all.tile(x1 - 1) + 1) * kTile > u.first;
                describe_columns<NT, 128 * NW>(a, u, b, h, rt, tree, sh.col, tid);
                if (tid < NT) {
                    const int r = rt * NT + tid, i = r / a.group;
                    const float lse =
                        i <= u.i1 ? a.lse_in[((size_t)b * a.n + i) * a.heads + h * a.group + r % a.group] : -INFINITY;
                    sh.col.less[tid] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
                }
                if (tid == 0) {
                    mbar_expect(&sh.q_ready, kQueryBytes<D, NT>);
                    load_queries<D, NT>(a, b, h, rt, sh.q[0], sh.col, &sh.q_ready);
                    sh.asked = seg + 1;
                }
                named_barrier<128 * NW>(3);
                if (tree) {
                    mark_kin<NT, 128 * NW>(sh.col, tid);
                    named_barrier<128 * NW>(3);
                }
                mbar_wait(&sh.q_ready, seg++ & 1, guard);
                for (int x = x0; x < x1; ++x) {
                    const int tile = all.tile(x);
                    if (!covers(u, tile))
                        continue;
                    if ((int)(g % NW) == w) {
                        // where a wait runs out, nothing came and nothing is added
                        bool came_all = mbar_wait(&sh.full[st], phase, guard);
                        const StageInfo &info = sh.info[st];
                        const int j0 = tile * kTile, j = j0 + t, page = info.page[t >> log_p];
                        const uint32_t came = came_all ? info.came : 0;
                        const bool edge = came != (1u << blocks) - 1 || !interior(a, u, j0);
                        const bool cached = !edge || (j < u.len && ((came >> (t >> log_p)) & 1));
                        const float ks = cached ? info.k_scale[t >> log_p] : 0.0f;
                        const float pos = FORM && a.f.slopes ? from_origin(a.c.positions ? info.pos[t] : j, sh.col.origin) : 0.0f;
                        const Mask<NT> see = edge && cached ? seen_by<NT>(a, askers, sh.col, j) : 0;
                        float *weight = a.weights + ((size_t)(cached ? page : 0) * a.c.kv_heads + h) * P + (t & (P - 1));
                        came_all = mbar_wait(&sh.s_full[w], (g / NW) & 1, guard) && came_all;
                        tc_after();
                        float sum = 0.0f;
#pragma unroll 1
                        for (int c0 = 0; c0 < NT; c0 += 16) {
                            alignas(8) float e[16];
                            alignas(8) float rest[16];
                            const uint32_t at = tmem + ((uint32_t)(wid & 3) << 21) + w * 2 * NT + c0;
                            TmemLoad<16>::go(at, e);
                            TmemLoad<16>::go(at + NT, rest);
                            tmem_wait<16>(e);
                            tmem_wait<16>(rest);
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                ((float2 *)e)[c] = add2(((float2 *)e)[c], ((float2 *)rest)[c]);
                            scores<FORM>(a, sh.col, sh.col.less, c0, ks, pos, e);
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                e[c] = exp2_fast(e[c]);
                            if (edge) {
                                const uint32_t bits = (uint32_t)(see >> c0);
#pragma unroll
                                for (int c = 0; c < 16; ++c)
                                    e[c] = (bits >> c) & 1 ? e[c] : 0.0f;
                            }
                            float2 *e2 = (float2 *)e;
#pragma unroll
                            for (int n = 4; n > 0; n >>= 1)
#pragma unroll
                                for (int c = 0; c < n; ++c)
                                    e2[c] = add2(e2[c], e2[c + n]);
                            sum += e[0] + e[1];
                        }
                        tc_before();
                        __syncwarp();
                        if (lane == 0 && came_all) {  // a tile that did not come is not given back
                            mbar_arrive(&sh.s_free[w]);
                            mbar_arrive(&sh.empty[st]);
                        }
                        // one addition a token and row tile, those of several row tiles a barrier apart: no order is left open,
                        // and nothing waits for the weight's old value
                        if (cached && came_all)
                            atomicAdd(weight, sum);
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
    tc_before();
    __syncthreads();
    tc_after();
    if (guard->dead) {
        if (wid == 0 && sh.asked > 0)
            land(&sh.q_ready, (sh.asked - 1) & 1);
        if (wid >= kProducer)  // the copies of this producer's last tiles
            for (int t = (int)sh.issued[wid - kProducer] - 1, k = 0; t >= 0 && k < ST; t -= 2, k += 2)
                land(&sh.full[t % ST], (t / ST) & 1);
        if (wid == kProducts)
            land_products(&sh.drained);
        if (tid == 0)
            report(a.status, SPEC_STATUS_INTERNAL);
        __syncthreads();
    }
    if (wid == kProducts)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Shared::kAlloc));
}

// Joins the parts of units that several CTAs worked on: a warp joins one row of
// the unit that ended in CTA blockIdx.x of attend_kernel, its lanes D / 32
// dimensions each (or, for the parts' totals, a part each).
constexpr int kJoinRows = 4;

template <int D, int NT> __global__ void __launch_bounds__(32 * kJoinRows) join_kernel(const __grid_constant__ AttendArgs a)
{
    using Vec = typename std::conditional<D == 128, float4, float2>::type;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int last = blockIdx.x, lane = threadIdx.x & 31;
    const int4 join = a.joins[last];
    if (join.x < 0)
        return;
    const int col = blockIdx.y * kJoinRows + (threadIdx.x >> 5), r = join.w * NT + col;
    if (r >= a.n * a.group)
        return;
    const auto slot = [&](int p) { return (2ll * p + (p == join.x)) * NT + col; };
    float top = -INFINITY;
    for (int p = join.x + lane; p <= last; p += 32) {
        const float2 s = a.part_sum[slot(p)];
        if (!(s.x == 0.0f))
            top = fmaxf(top, s.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // each part's output counts by its share of the total
    float total = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = join.x + lane; p <= last; p += 32) {
        const float2 s = a.part_sum[slot(p)];
        total += s.x == 0.0f ? 0.0f : s.x * exp2f(s.y - top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        total += __shfl_xor_sync(0xffffffffu, total, o);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll 4
    for (int p = join.x; p <= last; ++p) {
        const float2 s = a.part_sum[slot(p)];
        const Vec y = *(const Vec *)(a.part + slot(p) * D + lane * (D / 32));
        const bool some = !(s.x == 0.0f);
        const float w = s.x * exp2f(s.y - top) * inv;
        const float *v = (const float *)&y;
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
            o[k] += some ? v[k] * w : 0.0f;
    }
    const size_t row = ((size_t)join.y * a.n + r / a.group) * a.heads + join.z * a.group + r % a.group;
    __nv_bfloat162 *out = (__nv_bfloat162 *)(a.out + row * D + lane * (D / 32));
#pragma unroll
    for (int k = 0; k < D / 32; k += 2)
        out[k / 2] = __floats2bfloat162_rn(o[k], o[k + 1]);
    if (lane == 0)
        a.lse[row] = total == 0.0f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
}

// The kernels of one head size, by columns per row tile (16, 32 or 48).
struct Kernels {
    const void *split, *attend[3][2], *join[3], *weigh[3][2];  // [..][a cap or a bias]
    int attend_smem[3], attend_threads[3], weigh_smem[3];
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
    k.attend_threads[i] = AttendShape<D, NT>::kThreads;
    k.weigh_smem[i] = (int)sizeof(WeighShared<D, NT>) + 1024;
    static_assert(sizeof(AttendShared<D, NT>) + 2048 <= 227 * 1024 && sizeof(WeighShared<D, NT>) + 2048 <= 227 * 1024,
                  "shared memory of a CTA");
}
template <int D> Kernels all_kernels()
{
    Kernels k{};
    k.split = (const void *)split_kernel<D>;
    fill<D, 16>(k, 0);
    fill<D, 32>(k, 1);
    fill<D, 48>(k, 2);
    return k;
}

}  // namespace specc

#endif
