// spec_rows_product.cu -- rows times a weight's rows, both in 8 bits with scales of
// powers of two (spec_rows_product).  include/spec_verify.h states the operation.
//
//   out[t, n] = sum over blocks b of 2^(ea[t, b] + ew[n / 128, b]) * sum over the 128 k of b of a[t, k] w[n, k]
//
// A scale that is a power of two is what the tensor cores apply by themselves:
// tcgen05.mma kind::mxf8f6f4 takes one exponent byte for each row and 32 elements
// of either operand from tensor memory, so a block of 128 is four instructions with
// the same bytes, and the accumulator needs no pass through registers between
// blocks.  (With scales of any value each block's sums would have to be read from
// tensor memory, scaled and added: 128 x 240 values for every 64 instructions.)
//
// Two CTAs on neighbouring SMs work as a pair (cta_group::2): 256 of the weight's rows are the M side, 128 to each, and
// 32 to 240 of the activations' rows the N side, half of them brought by each.  (A round has few rows, which would fill
// a fraction of an M tile.)  A tile of 128 weight rows has one scale a block: all lanes of its columns hold the same
// word.  Four exponent bytes (four blocks, 512 elements of k) make one 32-bit column entry; the instruction descriptor
// says which byte is meant.
//
// Warps of a CTA: four that read accumulators and write the output, four that bring scales into tensor memory (each its
// 32 lanes), one for the copies and, in the first CTA of a pair, one that issues the products.
//
// Pairs are persistent, with accumulators in two places, so that writing one tile overlaps the products of the next.
// Where tiles are too few for the SMs, up to eight pairs share one, a part of k each.  Each CTA then adds up a share of the
// tile's rows, in the order of the parts, from what the others send into its shared memory (by bulk copies, which are faster
// than loads from theirs, 160 x 4,096 to 1,024 by 0.4 us, and than stores to its, by 2.5).  `plan` has the rule and what it
// rests on.
//
// Bound by the weight's bytes for few rows (1 x 4,096 to 128,256: 79.7 us, 98 % of the copy rate; 1 x 4,096 to 4,096: 6.9 us,
// of which more than 4 are this kernel's start and end), by the products for many (16,376 x 4,096 to 6,144: 196 to 213 us in
// short runs, 3.9 to 4.2 PFLOP/s, which a power limit lowers to 3.1 in long ones).  Without the scales' path that product took
// 190 us, without copies 177.  Few rows' times are of weights in memory; from L2 one row of 4,096 takes as long.

#include <algorithm>
#include <atomic>
#include <new>

#include "../cache/spec_ptx.cuh"
#include "spec_rows.cuh"

using namespace specc;

namespace {

constexpr int kRowsM = 128;   // weight rows of a CTA
constexpr int kMaxStages = 12;
constexpr int kThreads = 320;
constexpr int kScaleWarp = 4, kCopyWarp = 8, kIssueWarp = 9;
constexpr int kScaleColumns = 12;  // of one buffer: 4 for the weight's rows, 8 for up to 256 others
constexpr uint32_t kABytes = kRowsM * kScaleBlock;
constexpr uint32_t kChunkBytes = 32 * 32 * 2;  // outputs in bf16 that a warp writes together
constexpr int kOutRing = 4;                    // of them on their way
constexpr uint32_t kOutBytes = 4 * kOutRing * kChunkBytes;
constexpr int kDepth = 2;             // blocks of k to a stage
constexpr int kAhead = 4;             // of a CTA's first that it asks L2 for while the kernel before ends
constexpr uint32_t kColumns = 512;    // of tensor memory: all of them
constexpr int kMostRows = 240;        // of a tile: two accumulators and the scales take 504 columns
constexpr int kMaxSplits = 8;         // pairs that share a tile's k, in a cluster of twice as many CTAs

struct Args {
    const uint8_t *row_scale, *weight, *weight_scale;
    int64_t row_scale_stride, weight_stride, weight_scale_stride;
    void *out;
    int64_t out_stride;
    int rows, outs, blocks;  // activations' rows, weight rows, blocks of k
    int tile;                // activations' rows of a tile
    int row_tiles, out_tiles, group;
    int stages;
    uint32_t stage_bytes, b_bytes;
    uint32_t idesc;          // without the scales' bytes and the rows
    int splits, wide_out;    // wide_out: fp32
    int apart;               // other parts' sums arrive behind the stages, not in their place
    int boxes;               // outputs are written in boxes of 32 and 16 rows: 2 bf16, 4 fp32, 0 not
    int wait_limit;
    uint32_t *status;
};

// ---------------------------------------------------------------------------
// PTX that only these kernels use
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_index()
{
    uint32_t r;
    asm("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_count()
{
    uint32_t r;
    asm("mov.u32 %0, %%nclusterid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address of another CTA's shared memory, at the same place as `at` in this one's.
__device__ __forceinline__ uint32_t in_cluster(uint32_t at, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t in_cta(const void *p, uint32_t rank) { return in_cluster(smem_u32(p), rank); }
// From this CTA's shared memory to another's, whose barrier learns of the bytes.
__device__ __forceinline__ void copy_to(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "r"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ float4 load_shared4(uint32_t at)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
// For what went through tensor memory, which tcgen05.fence orders.  (A release at cluster scope, which nothing here needs,
// waits for the thread's loads in flight and more: 1,600 clocks each time.)
__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tell(int *flag, uint32_t rank)  // sets it in a CTA of the cluster
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_cta(flag, rank)), "r"(1) : "memory");
}
__device__ __forceinline__ void prefetch_line(const uint8_t *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory"); }
__device__ __forceinline__ void prefetch(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// What two CTAs do together: `mask` has a bit for the rank of each.
__device__ __forceinline__ void tmem_alloc(uint32_t *to, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(to)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t at, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}
__device__ __forceinline__ void commit(uint64_t *bar, uint32_t mask)  // in the CTAs of a pair
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "h"((uint16_t)mask)
                 : "memory");
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, bool add)
{
    asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %6, 0;\n"
                 "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
                 : "memory");
}
__device__ __forceinline__ void tma_load(const CUtensorMap *map, uint32_t dst, uint32_t bar, int k, int row)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, "
                 "%4}], [%2];" ::"r"(dst),
                 "l"(map), "r"(bar), "r"(k), "r"(row)
                 : "memory");
}

// mbar_wait for a whole warp: all of its lanes go on, or none does.
template <bool NOW = false> __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile Guard *guard)
{
    return __all_sync(0xffffffffu, mbar_wait<NOW>(bar, parity, guard));
}

// A place in a ring of buffers, and the parity of the phase that fills it this time round.
struct Ring {
    uint32_t at = 0, parity = 0;
    __device__ __forceinline__ void next(uint32_t size)
    {
        if (++at == size) {
            at = 0;
            parity ^= 1;
        }
    }
};

template <int N> __device__ __forceinline__ void tmem_store(uint32_t a, const uint32_t *u);
template <> __device__ __forceinline__ void tmem_store<4>(uint32_t a, const uint32_t *u)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0,%1,%2,%3};" ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(a)
                 : "memory");
}
template <> __device__ __forceinline__ void tmem_store<8>(uint32_t a, const uint32_t *u)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]),
                 "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(a)
                 : "memory");
}

// Ordinary loads, where they stand: the kernel ahead, which this one does not wait for before it begins, may be what writes
// the scales, so no load of them may promise constant memory.  (Written as *p they cost 167 registers instead of 126, and 1 to
// 3 %: 3 x 128 to 128,256 13.4 us against 12.4.)
__device__ __forceinline__ uint32_t load_byte(const uint8_t *p)
{
    uint32_t v;
    asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t load_word(const uint8_t *p)
{
    uint32_t v;
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint4 load_words(const uint8_t *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// A matrix of exponent bytes, from its first to behind its last.
struct Bytes {
    const uint8_t *begin, *end;
    bool aligned;  // rows at multiples of 16 bytes
    __device__ __forceinline__ Bytes(const uint8_t *p, int64_t stride, int64_t rows, int blocks)
        : begin(p), end(p + (rows - 1) * stride + blocks), aligned((((uint64_t)(uintptr_t)p | (uint64_t)stride) & 15) == 0)
    {
    }
    __device__ __forceinline__ uint32_t word(const uint8_t *p) const  // at a multiple of 4
    {
        if (p >= begin && p + 4 <= end)
            return load_word(p);
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (p + i >= begin && p + i < end)
                w |= load_byte(p + i) << 8 * i;
        return w;
    }
    // Blocks 16 q to 16 q + 15 of a row; behind the last block anything, which no instruction names.  Rows that begin
    // anywhere are read by aligned words, which may take in bytes of the row before or behind (333 x 2,832 to 5,000:
    // 12.9 us byte by byte, 12.3 so).  They are shifted into place when they are needed: until then loads are on their way.
    struct Sixteen {
        uint32_t w[5], shift;
        __device__ __forceinline__ uint4 get() const
        {
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = __funnelshift_r(w[i], w[i + 1], shift);
            return make_uint4(v[0], v[1], v[2], v[3]);
        }
    };
    __device__ __forceinline__ void blocks16(const uint8_t *row, int q, int blocks, Sixteen &s) const
    {
        const uint8_t *const p = row + 16 * q;
        const int left = blocks - 16 * q, off = (int)((uintptr_t)p & 3);
        s.shift = 8 * off;
        if (aligned && left >= 16) {
            const uint4 v = load_words(p);
            s.w[0] = v.x;
            s.w[1] = v.y;
            s.w[2] = v.z;
            s.w[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 5; ++i)
                if (4 * i < left + off)
                    s.w[i] = word(p - off + 4 * i);
        }
    }
};
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Unit u of the grid: `group` weight tiles beside each other share the activations' rows that pass through L2.
struct Tile {
    int out, row;
};
__device__ __forceinline__ Tile tile_of(const Args &a, int u)
{
    const int each = a.group * a.row_tiles, g = u / each, in = u - g * each;
    const int wide = min(a.group, a.out_tiles - g * a.group);
    return {g * a.group + in % wide, in / wide};
}

// Sixteen lanes (n) by 32 columns (rows t) of an accumulator, a pair of neighbouring columns in two registers: of the
// groups of eight columns the i-th is in v[4 i] to v[4 i + 3], lanes of the first half in the first two.
__device__ __forceinline__ void tmem_load_pairs(uint32_t at, float *v)
{
    uint32_t *const u = (uint32_t *)v;
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
                   "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
                 : "r"(at));
}
__device__ __forceinline__ uint32_t pack(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *(const uint32_t *)&h;
}
// Four 8 x 8 matrices of 16-bit values, transposed; lane i gives the address of row i % 8 of matrix i / 8.
__device__ __forceinline__ void store_transposed(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap *map, uint32_t src, int n, int row)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(n), "r"(row), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }

// Activations' rows that the products of a tile take: all of it, or as many as the last one has, in units of 16.
__device__ __forceinline__ int rows_of(const Args &a, const Tile &t) { return max(min(a.tile, (a.rows - t.row * a.tile + 15) & ~15), 32); }

__device__ __forceinline__ void store_shared(uint32_t at, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory"); }
__device__ __forceinline__ uint32_t load_shared(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
// Outputs of one type on their way to rows at any address: `rows` of them are staged together, `pitch` bytes apart (16 more
// than their values, so that eight rows lie in different banks).
template <typename T> struct Staged {
    static constexpr int rows = sizeof(T) == 2 ? 96 : 32;
    static constexpr uint32_t pitch = sizeof(T) * kRowsM + 16;
    static_assert(rows * pitch <= kOutBytes, "rows are staged in place of the boxes");
};
// Up to four rows of `width` outputs (128 at most) from shared memory to addresses that only their type aligns: a lane takes
// four values that lie together at a multiple of four, and eight lanes to a row the values before and behind those.
template <typename T> __device__ __forceinline__ void write_rows(T *to, int64_t stride, int count, int width, uint32_t from, int lane)
{
    constexpr int kWords = sizeof(T) == 2 ? 3 : 4;
    constexpr uint32_t kPitch = Staged<T>::pitch;
    const auto before = [](const T *p) { return (int)(-((uintptr_t)p / sizeof(T)) & 3); };
    uint32_t w[4][kWords];
    int first[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        first[j] = before(to + j * stride) + 4 * lane;
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            w[j][i] = load_shared(from + j * kPitch + (first[j] * (uint32_t)sizeof(T) & ~3u) + 4 * i);
    }
    const int j = lane / 8, k = lane & 7;
    T *const mine = to + j * stride;
    const int off = min(before(mine), width), at = k < 4 ? k : off + ((width - off) & ~3) + (k & 3);
    const uint32_t end = load_shared(from + j * kPitch + (at * (uint32_t)sizeof(T) & ~3u));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i < count && first[i] + 4 <= width) {
            T *const p = to + i * stride + first[i];
            if constexpr (sizeof(T) == 4)
                *(uint4 *)p = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
            else if (first[i] & 1)
                *(uint2 *)p = make_uint2(__funnelshift_r(w[i][0], w[i][1], 16), __funnelshift_r(w[i][1], w[i][2], 16));
            else
                *(uint2 *)p = make_uint2(w[i][0], w[i][1]);
        }
    }
    if (j < count && at < (k < 4 ? off : width)) {
        if constexpr (sizeof(T) == 4)
            *(uint32_t *)(mine + at) = end;
        else
            *(uint16_t *)(mine + at) = (uint16_t)(at & 1 ? end >> 16 : end);
    }
}

// 128 outputs of `used` rows by four warps, through shared memory at `at`: staged by all, then written a quarter each.
// acc: the warp's lanes of the accumulator.
template <typename T> __device__ __forceinline__ void write_tile(T *to, int64_t stride, int used, int width, uint32_t at, uint32_t acc, int warp, int lane)
{
    constexpr uint32_t kPitch = Staged<T>::pitch;
    for (int p = 0; p < used; p += Staged<T>::rows) {
        const int rows = min(Staged<T>::rows, used - p);
        for (int c = 0; c < rows; c += 32) {
            float v[32];
            if constexpr (sizeof(T) == 2) {
                tmem_load_pairs(acc + p + c, v);
                tmem_load_pairs(acc + (16u << 16) + p + c, v + 16);
                tmem_wait<32>(v);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    store_transposed(at + (c + 8 * i + (lane & 7)) * kPitch + warp * 64 + lane / 8 * 16, pack(v[4 * i], v[4 * i + 1]),
                                     pack(v[4 * i + 2], v[4 * i + 3]), pack(v[16 + 4 * i], v[17 + 4 * i]),
                                     pack(v[18 + 4 * i], v[19 + 4 * i]));
            } else {
                TmemLoad<16>::go(acc + p + c, v);
                TmemLoad<16>::go(acc + p + c + 16, v + 16);
                tmem_wait<32>(v);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    store_shared(at + (c + i) * kPitch + (warp * 32 + lane) * 4, v[i]);
            }
        }
        named_barrier<128>(2);
        for (int r = 4 * warp; r < rows && width > 0; r += 16)
            write_rows<T>(to + (p + r) * stride, stride, rows - r, width, at + r * kPitch, lane);
        named_barrier<128>(2);
    }
}

// Four neighbouring outputs of a row, together where the row lets them.
__device__ __forceinline__ void put4(const Args &a, int64_t row, int n, const float4 &v)
{
    const float e[4] = {v.x, v.y, v.z, v.w};
    if (a.wide_out) {
        float *const to = (float *)a.out + row * a.out_stride + n;
        if (n + 4 <= a.outs && ((uintptr_t)to & 15) == 0) {
            *(float4 *)to = v;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < a.outs)
                to[i] = e[i];
    } else {
        __nv_bfloat16 *const to = (__nv_bfloat16 *)a.out + row * a.out_stride + n;
        if (n + 4 <= a.outs && ((uintptr_t)to & 7) == 0) {
            *(uint2 *)to = make_uint2(pack(v.x, v.y), pack(v.z, v.w));
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < a.outs)
                to[i] = __float2bfloat16_rn(e[i]);
    }
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap rmap,
               const __grid_constant__ CUtensorMap omap)
{
    extern __shared__ uint8_t dynamic[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], scale_full[2], scale_empty[2], acc_full[2], acc_empty[2], ready, got, landed;
    __shared__ uint32_t tmem_at, scale_row[2][256];
    __shared__ Guard guard;
    uint8_t *const stage0 = (uint8_t *)(((uintptr_t)dynamic + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t side = rank & 1, leader = rank - side, mask = 3u << leader;  // of its pair
    const bool lead = side == 0;

    // blocks of k of this CTA
    const int part = (int)rank / 2;
    const int k0 = (int)((int64_t)a.blocks * part / a.splits), k1 = (int)((int64_t)a.blocks * (part + 1) / a.splits);
    const int units = a.row_tiles * a.out_tiles, step = (int)cluster_count();
    constexpr int kTileM = 2 * kRowsM;  // weight rows of a tile

    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&scale_full[i], 8);
            mbar_init(&scale_empty[i], 1);
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 8);
        }
        mbar_init(&ready, max(a.splits - 1, 1));
        mbar_init(&got, 1);
        mbar_init(&landed, 1);
        guard.dead = 0;
        guard.limit = a.wait_limit;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kCopyWarp) {
        if (elected()) {
            prefetch(&wmap);
            prefetch(&rmap);
        }
        __syncwarp();
        tmem_alloc(&tmem_at, kColumns);
    }
    tc_before();
    cluster_arrive();
    // L2 may begin to read the weight while the kernel before still runs: a hint, which brings nothing nearer than where
    // that kernel's writes arrive too, so it needs no promise that the weight stays.  A layer (width 4,096, one row):
    // 62.7 to 59.0 us; 1 x 4,096 to 4,096 behind itself: 7.9 to 6.9.  (As copies of tiles, or with more blocks than 4, what is
    // in L2 already costs more: 16 x 1,024 to 1,024 1.1 and 0.4 us.)  The warps that read accumulators have the time.
    // The first tile of this CTA, or the one that it has a part of, and the next one.  Found here, where there is time: divisions
    // take hundreds of clocks.
    const int u0 = (int)cluster_index();
    const Tile tile0 = tile_of(a, u0), tile1 = tile_of(a, min(u0 + step, units - 1));
    const int my_out = tile0.out * kTileM + (int)side * kRowsM, my_row = tile0.row * a.tile;
    if (warp < kScaleWarp) {
        const int n = my_out + threadIdx.x;
        const uint8_t *const p = a.weight + n * a.weight_stride;
        if (n < a.outs)
            for (int b = k0; b < min(k1, k0 + kAhead); ++b)
                prefetch_line(p + b * kScaleBlock);
    }
    // Where a tile's k is shared, each CTA adds up a share of the tile's rows; the other parts' sums of those arrive at `others`.
    const int my_used = min(a.tile, a.rows - my_row), share = (my_used + a.splits - 1) / a.splits, my_first = part * share,
              my_count = max(min(share, my_used - my_first), 0);
    const uint32_t others = smem_u32(stage0) + (a.apart ? a.stages * a.stage_bytes : my_used * (kRowsM * 4));
    asm volatile("griddepcontrol.wait;" ::: "memory");  // before any wait that is counted in clocks begins
    cluster_wait();
    tc_after();
    const uint32_t tmem = tmem_at, scales = tmem + kColumns - 2 * kScaleColumns;
    if (a.splits > 1 && threadIdx.x == 0)
        mbar_expect(&got, (a.splits - 1) * my_count * (kRowsM * 4));

    // A stage holds kDepth blocks of k.  The two loops below ask for the next barrier before they issue what the last one
    // allowed: a wait that begins when it is needed takes some 190 clocks even if there is nothing to wait for.
    if (warp == kCopyWarp) {
        Ring ring;
        uint32_t issued = 0;
        const uint32_t bar0 = in_cta(full, leader), base = smem_u32(stage0);
        bool free = true;
        for (int u = u0; u < units; u += step) {
            const Tile t = u == u0 ? tile0 : tile_of(a, u);
            const int n0 = t.out * kTileM + (int)side * kRowsM, r0 = t.row * a.tile + (int)side * (rows_of(a, t) / 2);
            for (int b = k0; b < k1; b += kDepth, ++issued) {
                if (!__all_sync(0xffffffffu, free) && !wait(&empty[ring.at], ring.parity ^ 1, &guard))
                    goto out;
                const uint32_t s = ring.at;
                ring.next(a.stages);
                free = mbar_test(&empty[ring.at], ring.parity ^ 1);
                if (elected()) {
                    const uint32_t at = base + s * a.stage_bytes, bar = bar0 + s * 8;
                    const int blocks = min(kDepth, k1 - b);
                    if (lead)
                        mbar_expect(&full[s], 2 * blocks * (kABytes + a.b_bytes));
#pragma unroll
                    for (int i = 0; i < kDepth; ++i)
                        if (i < blocks) {
                            tma_load(&wmap, at + i * kABytes, bar, (b + i) * kScaleBlock, n0);
                            tma_load(&rmap, at + kDepth * kABytes + i * a.b_bytes, bar, (b + i) * kScaleBlock, r0);
                        }
                }
                __syncwarp();
            }
        }
        // every stage given back: no arrival is on its way to this CTA's barriers when it ends
        for (int i = 0; i < a.stages; ++i) {
            if ((uint32_t)i < issued && !wait(&empty[i], ((issued - 1 - i) / a.stages) & 1, &guard))
                goto out;
        }
    } else if (warp == kIssueWarp && lead) {
        Ring ring;
        uint32_t groups = 0, done = 0;
        const uint32_t base = smem_u32(stage0);
        bool here = false, scaled = false;
        for (int u = u0; u < units; u += step, ++done) {
            const uint32_t buf = (done & 1), acc = tmem + buf * a.tile, n_bits = (uint32_t)rows_of(a, u == u0 ? tile0 : tile_of(a, u)) >> 3 << 17;
            if (!wait(&acc_empty[buf], (done >> 1 & 1) ^ 1, &guard))
                goto out;
            for (int b = k0; b < k1; b += kDepth) {
                const int blocks = min(kDepth, k1 - b);
                if (!__all_sync(0xffffffffu, here) && !wait(&full[ring.at], ring.parity, &guard))
                    goto out;
                const uint32_t s = ring.at;
                ring.next(a.stages);
                here = mbar_test(&full[ring.at], ring.parity);
#pragma unroll
                for (int i = 0; i < kDepth; ++i) {
                    const int k = b + i;
                    if (i < blocks) {
                        const uint32_t g = groups & 1;
                        if (k == k0 || (k & 3) == 0) {
                            if (!__all_sync(0xffffffffu, scaled) && !wait(&scale_full[g], groups >> 1 & 1, &guard))
                                goto out;
                            scaled = false;
                        } else if ((k & 3) == 3) {
                            scaled = mbar_test(&scale_full[g ^ 1], (groups + 1) >> 1 & 1);
                        }
                        tc_after();
                        const bool last = (k & 3) == 3 || k == k1 - 1;
                        if (elected()) {
                            const uint32_t at = base + s * a.stage_bytes;
                            // K-major, 128-byte rows in groups of eight; 32 elements further on are 32 bytes
                            const uint64_t da = smem_desc(at + i * kABytes, 16, 1024, 2),
                                           db = smem_desc(at + kDepth * kABytes + i * a.b_bytes, 16, 1024, 2);
                            const uint32_t id = a.idesc | n_bits | (uint32_t)(k & 3) << 4 | (uint32_t)(k & 3) << 29;
                            const uint32_t sa = scales + g * kScaleColumns;
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mma(acc, da + 2 * j, db + 2 * j, id, sa, sa + 4, k > k0 || j > 0);
                            if (i == blocks - 1)
                                commit(&empty[s], mask);
                            if (last)
                                commit(&scale_empty[g], mask);
                            if (k == k1 - 1)
                                commit(&acc_full[buf], mask);
                        }
                        __syncwarp();
                        groups += last;
                    }
                }
            }
        }
    } else if (warp >= kScaleWarp && warp < kScaleWarp + 4) {
        // A thread fetches the bytes of one or two rows, sixteen blocks or a tile ahead, once the word that is needed now has
        // been handed over (16,376 x 4,096 to 6,144: 199 us with a tile's first bytes fetched when it begins, 196 so; a fetch
        // ahead of that word makes narrow weights faster, 3 x 128 to 128,256 11.4 us against 12.1, and the first tile of all
        // slower, 160 x 1,024 to 28,672 11.3 against 10.9).  A word of each row goes through shared memory to the four warps,
        // which all store all rows (each for its 32 lanes, which the tensor cores read side by side).
        const int mine = threadIdx.x - kScaleWarp * 32;
        const uint32_t lanes = (uint32_t)(warp - kScaleWarp) << 21;  // 32 lanes of tensor memory each, at bit 16
        const Bytes row_bytes(a.row_scale, a.row_scale_stride, a.rows, a.blocks),
            weight_bytes(a.weight_scale, a.weight_scale_stride, (a.outs + kRowsM - 1) / kRowsM, a.blocks);
        // what is fetched next: of a tile that may be one ahead
        const uint8_t *wp, *p0, *p1;
        uint4 w, s0, s1;
        Bytes::Sixteen next_w{}, next0{}, next1{};
        const int last_wb = (a.outs - 1) / kRowsM;
        const auto turn = [&](const Tile &t) {
            // what has no row of its own reads the last one's bytes: they scale zeros that nothing is made of
            const int wb = min(t.out * 2 + (int)side, last_wb), r = t.row * a.tile + mine;
            wp = a.weight_scale + wb * a.weight_scale_stride;
            p0 = a.row_scale + min(r, a.rows - 1) * a.row_scale_stride;
            p1 = a.row_scale + min(r + 128, a.rows - 1) * a.row_scale_stride;
        };
        const auto fetch = [&](int q) {
            weight_bytes.blocks16(wp, q, a.blocks, next_w);
            row_bytes.blocks16(p0, q, a.blocks, next0);
            if (a.tile > 128)
                row_bytes.blocks16(p1, q, a.blocks, next1);
        };
        turn(tile0);
        fetch(k0 >> 4);
        Tile ahead = tile1;
        uint32_t groups = 0;
        w = s0 = s1 = make_uint4(0, 0, 0, 0);
        for (int u = u0; u < units; u += step) {
            for (int q = k0 >> 2; q <= (k1 - 1) >> 2; ++q, ++groups) {
                const uint32_t g = groups & 1;
                if (q == k0 >> 2 || (q & 3) == 0) {
                    w = next_w.get();
                    s0 = next0.get();
                    s1 = next1.get();
                }
                scale_row[g][mine] = word_of(s0, q & 3);
                if (a.tile > 128)
                    scale_row[g][mine + 128] = word_of(s1, q & 3);
                // the four warps agree on whether they go on: they meet at this barrier every time round
                if (barrier_or<128>(1, !wait(&scale_empty[g], (groups >> 1 & 1) ^ 1, &guard)))
                    goto out;
                tc_after();
                const uint32_t one = word_of(w, q & 3), same[4] = {one, one, one, one};
                uint32_t v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = i < 4 || a.tile > 128 ? scale_row[g][32 * i + lane] : 0;
                const uint32_t at = scales + g * kScaleColumns + lanes;
                tmem_store<4>(at, same);
                if (a.tile > 128)
                    tmem_store<8>(at + 4, v);
                else
                    tmem_store<4>(at + 4, v);
                tmem_store_wait();
                tc_before();
                __syncwarp();
                if (lane == 0)
                    arrive_cluster(in_cta(&scale_full[g], leader));
                if (q == k0 >> 2 || (q & 3) == 0) {
                    if (16 * ((q >> 2) + 1) < k1) {
                        fetch((q >> 2) + 1);
                    } else if (u + step < units) {
                        turn(ahead);
                        fetch(k0 >> 4);
                    }
                }
            }
            ahead = tile_of(a, min(u + 2 * step, units - 1));
        }
        for (uint32_t i = groups > 2 ? groups - 2 : 0; i < groups; ++i)
            if (!wait(&scale_empty[i & 1], i >> 1 & 1, &guard))
                goto out;
    } else if (warp < kScaleWarp) {
        const uint32_t lanes = (uint32_t)warp << 21, chunk0 = smem_u32(stage0) + a.stages * a.stage_bytes + warp * (kOutRing * kChunkBytes);
        uint32_t done = 0, chunks = 0;
        // what a lane sends to the part of its number, if there is one
        const bool sends = lane < a.splits && lane != part;
        const uint32_t other = 2 * lane + side, bytes = max(min(share, my_used - lane * share), 0) * (kRowsM * 4),
                       to = in_cluster(others + (part - (part > lane)) * share * (kRowsM * 4), sends ? other : rank),
                       bar = in_cta(&got, sends ? other : rank);
        for (int u = u0; u < units; u += step, ++done) {
            const Tile t = u == u0 ? tile0 : tile_of(a, u);
            const uint32_t buf = (done & 1), acc = tmem + buf * a.tile + lanes;
            const int m = warp * 32 + lane, n = t.out * kTileM + (int)side * kRowsM + m, r0 = t.row * a.tile;
            const int used = min(a.tile, a.rows - r0);
            if (barrier_or<128>(2, !wait<true>(&acc_full[buf], done >> 1 & 1, &guard)))
                goto out;
            tc_after();
            if (a.boxes == 2) {
                // 32 outputs and up to 32 rows at a time, transposed on their way through shared memory; the next ones are
                // on their way from tensor memory meanwhile, and up to kOutRing of them to global memory
                const auto load = [&](int c, float *v) {
                    tmem_load_pairs(acc + c, v);
                    tmem_load_pairs(acc + (16u << 16) + c, v + 16);
                };
                const auto write = [&](int c, const float *v) {
                    const uint32_t at = chunk0 + (chunks++ % kOutRing) * kChunkBytes;
                    if (lane == 0)
                        store_wait_read<kOutRing - 1>();
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // matrix j of the four: weight rows 8 j to 8 j + 7 of the warp's, activations' rows 8 i to 8 i + 7
                        const int row = 8 * i + (lane & 7);
                        store_transposed(at + row * 64 + ((lane / 8 ^ (row >> 1 & 3)) << 4), pack(v[4 * i], v[4 * i + 1]),
                                         pack(v[4 * i + 2], v[4 * i + 3]), pack(v[16 + 4 * i], v[17 + 4 * i]),
                                         pack(v[18 + 4 * i], v[19 + 4 * i]));
                    }
                    proxy_fence();
                    __syncwarp();
                    if (lane == 0) {
                        // boxes of 32 outputs and 16 rows, those that begin inside the tile and the output
                        if (n < a.outs) {
                            tma_store(&omap, at, n, r0 + c);
                            if (c + 16 < used)
                                tma_store(&omap, at + kChunkBytes / 2, n, r0 + c + 16);
                        }
                        store_commit();
                    }
                };
                float v[32], w[32];
                load(0, v);
                for (int c = 0; c < used; c += 64) {
                    tmem_wait<32>(v);
                    if (c + 32 < used)
                        load(c + 32, w);
                    write(c, v);
                    if (c + 32 >= used)
                        break;
                    tmem_wait<32>(w);
                    if (c + 64 < used)
                        load(c + 64, v);
                    write(c + 32, w);
                }
            } else if (a.boxes == 4) {
                for (int c = 0; c < used; c += 32, ++chunks) {
                    float v[32];
                    TmemLoad<16>::go(acc + c, v);
                    TmemLoad<16>::go(acc + c + 16, v + 16);
                    const uint32_t at = chunk0 + (chunks & 1) * (2 * kChunkBytes);
                    if (lane == 0)
                        store_wait_read<1>();
                    __syncwarp();
                    tmem_wait<32>(v);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        store_shared(at + i * 128 + lane * 4, v[i]);
                    proxy_fence();
                    __syncwarp();
                    if (lane == 0) {
                        if (n < a.outs) {
                            tma_store(&omap, at, n, r0 + c);
                            if (c + 16 < used)
                                tma_store(&omap, at + kChunkBytes, n, r0 + c + 16);
                        }
                        store_commit();
                    }
                }
            } else if (a.splits > 1) {
                // the copies into the stages have all been used by now, in whose place the sums go
                if (!a.apart && warp == 0 && sends)
                    arrive_cluster(in_cta(&ready, other));
                const uint32_t at = smem_u32(stage0) + m * 4;
                for (int c = 0; c < used; c += 32) {
                    float v[32];
                    TmemLoad<16>::go(acc + c, v);
                    TmemLoad<16>::go(acc + c + 16, v + 16);
                    tmem_wait<32>(v);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c + i < used)
                            store_shared(at + (c + i) * (kRowsM * 4), v[i]);
                }
                proxy_fence();
                named_barrier<128>(2);
                if (warp == 0 && (a.apart || wait(&ready, 0, &guard)) && sends && bytes)
                    copy_to(to, smem_u32(stage0) + lane * share * (kRowsM * 4), bytes, bar);
            } else {
                // Rows at any address (bf16, 16,384 x 64 to 12,207: 307 us with single values from the registers, 244 so; 131
                // in boxes)
                const uint32_t at = smem_u32(stage0) + a.stages * a.stage_bytes;
                const int64_t begin = r0 * a.out_stride + (n - m);
                const int width = min(kRowsM, a.outs - (n - m));
                if (a.wide_out)
                    write_tile((float *)a.out + begin, a.out_stride, used, width, at, acc, warp, lane);
                else
                    write_tile((__nv_bfloat16 *)a.out + begin, a.out_stride, used, width, at, acc, warp, lane);
            }
            tc_before();
            __syncwarp();
            if (lane == 0 && u + 2 * step < units)  // where a tile is yet to come that waits for it
                arrive_cluster(in_cta(&acc_empty[buf], leader));
        }
    }
out:
    // The next kernel's CTAs need this one's shared memory; begun any earlier they wait beside it (212 to 225 us against 200
    // for 16,376 x 4,096 to 6,144).
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp < kScaleWarp && lane == 0)
        store_wait_read<0>();  // the buffers are the CTA's for as long as copies read them
    __syncwarp();
    if (a.splits > 1) {
        __syncthreads();
        if (wait(&got, 0, &guard) && my_out + lane * 4 < a.outs) {
            const uint32_t at = lane * 16, own = smem_u32(stage0) + my_first * (kRowsM * 4) + at;
            constexpr int kWarps = kThreads / 32, kMore = 4;  // rows whose loads are in flight together
            for (int r = warp; r < my_count; r += kWarps * kMore) {
                float4 sum[kMore];
#pragma unroll
                for (int i = 0; i < kMore; ++i)
                    sum[i] = make_float4(0, 0, 0, 0);
                for (int k = 0; k < a.splits; ++k) {  // in the order of the parts
                    const uint32_t from = (k == part ? own : others + at + (k - (k > part)) * share * (kRowsM * 4)) + r * (kRowsM * 4);
                    float4 v[kMore];
#pragma unroll
                    for (int i = 0; i < kMore; ++i)
                        v[i] = r + i * kWarps < my_count ? load_shared4(from + i * (kWarps * kRowsM * 4)) : make_float4(0, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < kMore; ++i) {
                        sum[i].x += v[i].x;
                        sum[i].y += v[i].y;
                        sum[i].z += v[i].z;
                        sum[i].w += v[i].w;
                    }
                }
#pragma unroll
                for (int i = 0; i < kMore; ++i)
                    if (r + i * kWarps < my_count)
                        put4(a, my_row + my_first + r + i * kWarps, my_out + lane * 4, sum[i]);
            }
        }
    }
    const bool dead = __syncthreads_or(guard.dead);
    if (dead) {
        if (warp == kIssueWarp && lead && elected()) {  // the products in flight
            commit(&landed, mask);
            land(&landed, 0);
        }
        if (threadIdx.x == 0)
            report(a.status, SPEC_STATUS_INTERNAL);
        if (threadIdx.x < 2 * a.splits)
            tell(&guard.dead, threadIdx.x);
        __syncwarp();
    }
    tc_before();
    // All that was sent to another CTA and its barriers has been waited for there, unless a wait ran out: so this need not wait
    // for the outputs on their way (1 x 4,096 to 4,096: 7.3 us if it does, 6.9 so).
    if (dead)
        cluster_arrive();
    else
        cluster_arrive_relaxed();
    cluster_wait();
    tc_after();
    if (warp == kCopyWarp)
        tmem_dealloc(tmem, kColumns);
    // If a wait ran out in any CTA of the cluster, what is in flight between them and into them lands before the memory of one
    // is given back.  No barrier tells of it (a stage that only one CTA of a pair filled never completes its phase), so each
    // waits out a time that a copy takes many times over.
    if (threadIdx.x == 0 && ((volatile Guard &)guard).dead) {
        const long long since = clock64();
        while (clock64() - since < (1 << 22))
            ;
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
struct Device {
    int sms = 0;
    int clusters[kMaxSplits + 1] = {};  // clusters of 2 n CTAs that run at once
};

// Dynamic shared memory: nearly all of it.  A CTA holds all of tensor memory, so nothing else that waits for some may be
// on its SM, where two clusters could each hold what the other waits for.
constexpr uint32_t kShared = 223 * 1024;

constexpr uint32_t stage_bytes(int tile) { return kDepth * (kABytes + (uint32_t)(tile / 2) * kScaleBlock); }
// What arrives from the other parts.
constexpr uint32_t others_bytes(int tile, int parts) { return (uint32_t)((parts - 1) * ((tile + parts - 1) / parts)) * kRowsM * 4; }
// They have their own place while that costs no stage that is missed; in the place of stages they must wait until that CTA
// has used them (14 x 14,336 to 1: 7.05 us apart, 7.2 not; 160 x 8,192 to 8,192: 17.3 us apart, 16.4 not).
constexpr bool others_apart(int tile, int parts) { return parts > 1 && tile <= 64; }
// Stages, beside the outputs on their way or what arrives from the other parts.
constexpr int stages_of(int tile, int parts)
{
    const uint32_t beside = parts == 1 ? kOutBytes : others_apart(tile, parts) ? others_bytes(tile, parts) : 0;
    return (int)std::min<uint32_t>(kMaxStages, (kShared - 1024 - beside) / stage_bytes(tile));
}

struct Plan {
    int tile, splits;
};

// The tile and the parts of k of least estimated time.  In units of 0.1 ns: a block of k takes 185 ns + 0.6 a row of the
// tile (issue, then copies and products; 32 blocks of 16,376 rows to 6,144: 6.5 us with 32 rows, 9.7 with 240), in as many
// rounds as there are tiles to a pair of SMs; adding up n parts takes 0.1 us and n times 40 ns + 3 a row (one row of 14,336
// to one output: 27.7 us whole, 15.7, 9.6 and 7.1 in 2, 4 and 8 parts), and each pair at work 15 ns more, as they start together
// and meet.  Parts that do not all run at once cost a round more than they save (256 rows of 2,048 to 2,048, 64 rows to a
// tile: 7.0 us whole, 7.1 in two parts, 12.8 in three).  Over 108 sizes the choice is within 4 % of the best of them in 102
// and within 10 % in all but one (640 to 4,096, 128 rows: 5.6 us, 5.0 in tiles of 64 rows).  It does not look at where outputs
// lie, nor at what writing them takes.
Plan plan(const Device &d, int rows, int outs, int blocks)
{
    const int64_t out_tiles = (outs + 2 * kRowsM - 1) / (2 * kRowsM);
    Plan p{};
    int64_t best = INT64_MAX;
    for (int tile = 32; tile <= kMostRows; tile += 16) {
        const int64_t units = out_tiles * ((rows + tile - 1) / tile), rounds = (units + d.sms / 2 - 1) / (d.sms / 2);
        for (int n = 1; n <= kMaxSplits; ++n) {
            if (n > 1 && (units > d.clusters[n] || n > blocks || (uint32_t)tile * kRowsM * 4 + others_bytes(tile, n) > kShared - 1024))
                break;
            const int64_t each = (blocks + n - 1) / n * (1850 + 6 * tile);
            const int64_t cost = n == 1 ? rounds * each : each + 1000 + n * (400 + 30 * tile + 150 * units);
            if (cost < best) {
                best = cost;
                p = {tile, n};
            }
        }
        if (tile >= rows)
            break;
    }
    return p;
}

constexpr int kMaxDevices = 64;
std::atomic<const Device *> g_devices[kMaxDevices];  // made once each, and kept

spec_status this_device(const Device **out)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return SPEC_ERR_CUDA;
    }
    if (dev < 0 || dev >= kMaxDevices)
        return SPEC_ERR_UNSUPPORTED;
    const Device *found = g_devices[dev].load(std::memory_order_acquire);
    if (!found) {
        Device d;
        if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaFuncSetAttribute(product_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared) != cudaSuccess ||
            cudaFuncSetAttribute(product_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
            cudaGetLastError();
            return SPEC_ERR_CUDA;
        }
        for (int n = 1; n <= kMaxSplits; ++n) {
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2 * n;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(2 * n * d.sms);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = kShared;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&d.clusters[n], product_kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();
                return SPEC_ERR_CUDA;
            }
        }
        if (d.sms < 2 || d.clusters[1] < 1)
            return SPEC_ERR_UNSUPPORTED;
        Device *const made = new (std::nothrow) Device(d);
        if (!made)
            return SPEC_ERR_CUDA;
        found = nullptr;
        if (!g_devices[dev].compare_exchange_strong(found, made, std::memory_order_acq_rel))
            delete made;  // another thread was first
        else
            found = made;
    }
    *out = found;
    return SPEC_OK;
}

// [element, row], rows `stride` bytes apart; a box is box_bytes of box_rows rows.
spec_status make_map(CUtensorMapDataType type, int element, int box_bytes, CUtensorMapSwizzle swizzle, void *at, int64_t dim, int64_t rows,
                     int64_t stride, int box_rows, CUtensorMap *map)
{
    const EncodeTiled encode = encoder();
    if (!encode)
        return SPEC_ERR_CUDA;
    const cuuint64_t size[2] = {(cuuint64_t)dim, (cuuint64_t)rows}, step[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {(cuuint32_t)(box_bytes / element), (cuuint32_t)box_rows}, one[2] = {1, 1};
    return encode(map, type, 2, at, size, step, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? SPEC_OK
               : SPEC_ERR_INVALID_ARG;
}
spec_status make_map(const spec_coded *c, int box_rows, CUtensorMap *map)
{
    return make_map(CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128, CU_TENSOR_MAP_SWIZZLE_128B, c->codes, c->dim, c->rows, c->stride, box_rows, map);
}

}  // namespace

extern "C" spec_status spec_rows_product(const spec_coded *rows, const spec_coded *weight, void *out, int64_t out_stride,
                                         spec_dtype dtype, uint32_t *status, void *stream)
{
    NvtxScope nvtx("spec_rows_product");
    spec_status st = check_coded(rows);
    if (st == SPEC_OK)
        st = check_coded(weight);
    if (st != SPEC_OK)
        return st;
    if (bad_dtype(dtype))
        return SPEC_ERR_UNSUPPORTED;
    if (rows->dim != weight->dim)
        return SPEC_ERR_INVALID_ARG;
    if (rows->rows == 0 || weight->rows == 0)
        return SPEC_OK;
    const int64_t size = dtype == SPEC_BF16 ? 2 : 4;
    if (!out || ((uintptr_t)out & (size - 1)) || out_stride < weight->rows || out_stride >= (1ll << 38) || bad4(status, false))
        return SPEC_ERR_INVALID_ARG;
    const Device *device = nullptr;
    st = this_device(&device);
    if (st != SPEC_OK)
        return st;
    Args a{};
    a.row_scale = rows->scale;
    a.row_scale_stride = rows->scale_stride;
    a.weight = (const uint8_t *)weight->codes;
    a.weight_stride = weight->stride;
    a.weight_scale = weight->scale;
    a.weight_scale_stride = weight->scale_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.rows = rows->rows;
    a.outs = weight->rows;
    a.blocks = scale_blocks(rows->dim);
    const Plan p = plan(*device, a.rows, a.outs, a.blocks);
    a.tile = p.tile;
    a.splits = p.splits;
    a.row_tiles = (a.rows + p.tile - 1) / p.tile;
    a.out_tiles = (a.outs + 2 * kRowsM - 1) / (2 * kRowsM);
    if ((int64_t)a.row_tiles * a.out_tiles > INT_MAX / (2 * kMaxSplits))
        return SPEC_ERR_UNSUPPORTED;
    // Eight weight tiles side by side share the rows that pass through L2; as many as stay there (32 MB of them) where the
    // rows themselves do not, so that those pass once (16,376 x 4,096 to 6,144: 224 us with 8, 197 with all 24; 1,280 x
    // 4,096 to 128,256: 395 us with 8, 440 with 64).
    a.group = 8;
    if ((int64_t)a.rows * a.blocks > (16 << 20) / kScaleBlock)
        a.group = std::max(8, (int)std::min<int64_t>(a.out_tiles, (32 << 20) / ((int64_t)2 * kRowsM * kScaleBlock * a.blocks)));
    a.b_bytes = (uint32_t)(p.tile / 2) * kScaleBlock;  // a multiple of 1,024
    a.stage_bytes = stage_bytes(p.tile);
    a.boxes = p.splits == 1 && ((uintptr_t)out & 15u) == 0 && (out_stride * size & 15) == 0 ? (int)size : 0;
    a.stages = stages_of(p.tile, p.splits);
    a.apart = others_apart(p.tile, p.splits);
    // as in the unscaled kinds, and: bytes of the scales at bits 4 and 29 (set for each block, as the rows at bit 17 are for each tile), scales of powers of
    // two (bit 23)
    a.idesc = (uint32_t)(weight->code == SPEC_E5M2) << 7 | (uint32_t)(rows->code == SPEC_E5M2) << 10 |
              1u << 23 | (uint32_t)(2 * kRowsM >> 7) << 27;
    a.wide_out = dtype == SPEC_F32;
    a.wait_limit = wait_limit();
    a.status = status;
    CUtensorMap wmap, rmap, omap{};
    if ((st = make_map(weight, kRowsM, &wmap)) != SPEC_OK || (st = make_map(rows, p.tile / 2, &rmap)) != SPEC_OK ||
        (a.boxes &&
         (st = dtype == SPEC_BF16
                   ? make_map(CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, 64, CU_TENSOR_MAP_SWIZZLE_64B, out, a.outs, a.rows, out_stride * 2, 16, &omap)
                   : make_map(CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, 128, CU_TENSOR_MAP_SWIZZLE_NONE, out, a.outs, a.rows, out_stride * 4, 16,
                              &omap)) != SPEC_OK))
        return st;
    const int units = a.row_tiles * a.out_tiles;
    const dim3 grid((unsigned)(2 * p.splits * (p.splits == 1 ? std::min(units, device->sms / 2) : units)));
    return launch(product_kernel, grid, kThreads, kShared, 2 * p.splits, (cudaStream_t)stream, a, wmap, rmap, omap);
}
