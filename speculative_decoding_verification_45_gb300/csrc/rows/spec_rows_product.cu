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
// The weight's rows are the M side (128 to a CTA), the activations' rows the N side
// (16 to 240): a round has few rows, which would fill a fraction of an M tile.  A
// tile of 128 weight rows has one scale a block: all lanes of its column hold the
// same word.  Four exponent bytes (four blocks, 512 elements of k) make one 32-bit
// column entry; the instruction descriptor says which byte is meant.
//
// Warps of a CTA: four that read accumulators and write the output, four that bring
// scales into tensor memory (each its 32 lanes), one for the copies, one that issues
// the products.
//
// Two arrangements (the rule is at `plan`):
//   pair    two CTAs share tiles of 256 weight rows; each brings half of the other
//           operand (cta_group::2).  Persistent, accumulators in two halves of tensor
//           memory, so that writing one tile overlaps the products of the next.
//   split   a tile for each cluster; its CTAs take equal parts of k and add their
//           sums through distributed shared memory, in the order of their ranks.

#include <algorithm>
#include <atomic>

#include "../spec_ptx.cuh"
#include "spec_rows.cuh"

using namespace specc;

namespace {

constexpr int kRowsM = 128;   // weight rows of a CTA
// Two accumulators of up to 240 rows and the scales fill 504 of the 512 columns of tensor memory.
constexpr int kMaxStages = 12;
constexpr int kThreads = 320;
constexpr int kScaleWarp = 4, kCopyWarp = 8, kIssueWarp = 9;
constexpr int kScaleColumns = 12;  // of one buffer: 4 for the weight's rows, 8 for up to 256 others
constexpr uint32_t kABytes = kRowsM * kScaleBlock;
constexpr int kChunk = 32;  // activations' rows that are written together
constexpr uint32_t kChunkBytes = kChunk * kRowsM * 2;

struct Args {
    const uint8_t *row_scale, *weight_scale;
    int64_t row_scale_stride, weight_scale_stride;
    void *out;
    int64_t out_stride;
    int rows, outs, blocks;  // activations' rows, weight rows, blocks of k
    int tile;                // activations' rows of a tile
    int row_tiles, out_tiles, group;
    int stages;
    uint32_t stage_bytes, b_bytes;
    uint32_t columns;        // of tensor memory
    uint32_t idesc;          // without the scales' bytes
    int splits, wide_out;    // wide_out: fp32
    int tma_out;             // bf16 rows at multiples of 16 bytes
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
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of another CTA's shared memory, at the same place as `p` in this one's.
__device__ __forceinline__ uint32_t in_cta(const void *p, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ float load_cluster(uint32_t a)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
// For what went through tensor memory, which tcgen05.fence orders.  (A release at cluster scope, which nothing here needs,
// waits for the thread's loads in flight and more: 1,600 clocks each time, 311 us against 290 for 16,376 x 4,096 to 6,144.)
__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <int CG> struct Pair;
template <> struct Pair<1> {
    static __device__ __forceinline__ void alloc(uint32_t *to, uint32_t columns)
    {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(to)), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    static __device__ __forceinline__ void dealloc(uint32_t at, uint32_t columns)
    {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
    }
    static __device__ __forceinline__ void commit(uint64_t *bar) { tc_commit(bar); }
    static __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, bool add)
    {
        asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %6, 0;\n"
                     "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
                     : "memory");
    }
    static __device__ __forceinline__ void load(const CUtensorMap *map, uint32_t dst, uint32_t bar, int k, int row)
    {
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                         dst),
                     "l"(map), "r"(bar), "r"(k), "r"(row)
                     : "memory");
    }
};
template <> struct Pair<2> {
    static __device__ __forceinline__ void alloc(uint32_t *to, uint32_t columns)
    {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(to)), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    static __device__ __forceinline__ void dealloc(uint32_t at, uint32_t columns)
    {
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
    }
    static __device__ __forceinline__ void commit(uint64_t *bar)  // in both CTAs
    {
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                         smem_u32(bar)),
                     "h"((uint16_t)3)
                     : "memory");
    }
    static __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, bool add)
    {
        asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %6, 0;\n"
                     "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
                     : "memory");
    }
    static __device__ __forceinline__ void load(const CUtensorMap *map, uint32_t dst, uint32_t bar, int k, int row)
    {
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, "
                     "%4}], [%2];" ::"r"(dst),
                     "l"(map), "r"(bar), "r"(k), "r"(row)
                     : "memory");
    }
};

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

// Exponent bytes of blocks 16 q to 16 q + 15 of a row, in one load where row and bytes allow; 1 behind the last block (no
// instruction names those).
__device__ __forceinline__ uint4 scale_words(const uint8_t *row, int q, int blocks, int aligned)
{
    uint32_t w[4];
    const uint8_t *const p = row + 16 * q;
    if (aligned == 16 && 16 * q + 16 <= blocks)
        return __ldg((const uint4 *)p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int left = blocks - 16 * q - 4 * i;
        w[i] = 0x7f7f7f7fu;
        if (aligned >= 4 && left >= 4) {
            w[i] = __ldg((const uint32_t *)(p + 4 * i));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < left)
                    w[i] = (w[i] & ~(0xffu << 8 * j)) | (uint32_t)__ldg(p + 4 * i + j) << 8 * j;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ int alignment_of(const uint8_t *p, int64_t stride)
{
    const uint64_t u = (uint64_t)(uintptr_t)p | (uint64_t)stride;
    return (u & 15) == 0 ? 16 : (u & 3) == 0 ? 4 : 1;
}
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

__device__ __forceinline__ void put(const Args &a, int64_t row, int col, float v)
{
    if (a.wide_out)
        ((float *)a.out)[row * a.out_stride + col] = v;
    else
        ((__nv_bfloat16 *)a.out)[row * a.out_stride + col] = __float2bfloat16_rn(v);
}

// Blocks of k to a stage.
template <int CG> struct Depth {
    static constexpr int value = CG;
};

// ---------------------------------------------------------------------------
// The kernel.  CG: CTAs that issue products together.
// ---------------------------------------------------------------------------
template <int CG> __global__ void __launch_bounds__(kThreads, CG == 1 ? 2 : 1)
product_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap rmap,
               const __grid_constant__ CUtensorMap omap)
{
    extern __shared__ uint8_t dynamic[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], scale_full[2], scale_empty[2], acc_full[2], acc_empty[2], landed;
    __shared__ uint32_t tmem_at, scale_row[2][256];
    __shared__ Guard guard;
    uint8_t *const stage0 = (uint8_t *)(((uintptr_t)dynamic + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool lead = CG == 1 || rank == 0;
    const bool linked = CG == 2 || a.splits > 1;
    constexpr int kDepth = Depth<CG>::value;
    constexpr int kBuffers = CG;  // accumulators: a CTA of a split has one tile

    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&scale_full[i], 4 * CG);
            mbar_init(&scale_empty[i], 1);
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4 * CG);
        }
        mbar_init(&landed, 1);
        guard.dead = 0;
        guard.limit = a.wait_limit;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kCopyWarp)
        Pair<CG>::alloc(&tmem_at, a.columns);
    tc_before();
    if (linked)
        cluster_sync();
    else
        __syncthreads();
    tc_after();
    const uint32_t tmem = tmem_at, scales = tmem + a.columns - 2 * kScaleColumns;

    // blocks of k of this CTA
    const int part = CG == 1 ? (int)rank : 0;
    const int k0 = (int)((int64_t)a.blocks * part / a.splits), k1 = (int)((int64_t)a.blocks * (part + 1) / a.splits);
    const int units = a.row_tiles * a.out_tiles, step = (int)cluster_count();
    const int own_rows = CG * kRowsM;  // weight rows of a tile

    // A stage holds kDepth blocks of k.  The two loops below ask for the next barrier before they issue what the last one
    // allowed: a wait that begins when it is needed takes some 190 clocks even if there is nothing to wait for.
    if (warp == kCopyWarp) {
        Ring ring;
        uint32_t issued = 0;
        const uint32_t bar0 = CG == 1 ? smem_u32(full) : in_cta(full, 0), base = smem_u32(stage0);
        bool free = true;
        for (int u = (int)cluster_index(); u < units; u += step) {
            const Tile t = tile_of(a, u);
            const int n0 = t.out * own_rows + (CG == 2 ? (int)rank * kRowsM : 0), r0 = t.row * a.tile + (CG == 2 ? (int)rank * (a.tile / 2) : 0);
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
                        mbar_expect(&full[s], CG * blocks * (kABytes + a.b_bytes));
#pragma unroll
                    for (int i = 0; i < kDepth; ++i)
                        if (i < blocks) {
                            Pair<CG>::load(&wmap, at + i * kABytes, bar, (b + i) * kScaleBlock, n0);
                            Pair<CG>::load(&rmap, at + kDepth * kABytes + i * a.b_bytes, bar, (b + i) * kScaleBlock, r0);
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
        for (int u = (int)cluster_index(); u < units; u += step, ++done) {
            const uint32_t buf = done % kBuffers, acc = tmem + buf * a.tile;
            if (!wait(&acc_empty[buf], (done / kBuffers & 1) ^ 1, &guard))
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
                            const uint32_t id = a.idesc | (uint32_t)(k & 3) << 4 | (uint32_t)(k & 3) << 29;
                            const uint32_t sa = scales + g * kScaleColumns;
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                Pair<CG>::mma(acc, da + 2 * j, db + 2 * j, id, sa, sa + 4, k > k0 || j > 0);
                            if (i == blocks - 1)
                                Pair<CG>::commit(&empty[s]);
                            if (last)
                                Pair<CG>::commit(&scale_empty[g]);
                            if (k == k1 - 1)
                                Pair<CG>::commit(&acc_full[buf]);
                        }
                        __syncwarp();
                        groups += last;
                    }
                }
            }
        }
    } else if (warp >= kScaleWarp && warp < kScaleWarp + 4) {
        // A thread fetches the bytes of one or two rows, sixteen blocks ahead; a word of each goes through shared memory to
        // the four warps, which all store all rows (each for its 32 lanes, which the tensor cores read side by side).
        const int mine = threadIdx.x - kScaleWarp * 32;
        const uint32_t lanes = (uint32_t)(warp - kScaleWarp) << 21;  // 32 lanes of tensor memory each, at bit 16
        const int row_aligned = alignment_of(a.row_scale, a.row_scale_stride), weight_aligned = alignment_of(a.weight_scale, a.weight_scale_stride);
        const uint4 one4 = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
        uint32_t groups = 0;
        for (int u = (int)cluster_index(); u < units; u += step) {
            const Tile t = tile_of(a, u);
            const int wb = t.out * CG + (CG == 2 ? (int)rank : 0), r0 = t.row * a.tile;
            const bool has = (int64_t)wb * kRowsM < a.outs, has0 = mine < a.tile && r0 + mine < a.rows,
                       has1 = mine + 128 < a.tile && r0 + mine + 128 < a.rows;
            const uint8_t *const wp = a.weight_scale + wb * a.weight_scale_stride,
                                *const p0 = a.row_scale + (r0 + mine) * a.row_scale_stride, *const p1 = p0 + 128 * a.row_scale_stride;
            uint4 w, s0, s1, next_w, next0, next1;
            const auto fetch = [&](int q) {
                next_w = has ? scale_words(wp, q, a.blocks, weight_aligned) : one4;
                next0 = has0 ? scale_words(p0, q, a.blocks, row_aligned) : one4;
                next1 = has1 ? scale_words(p1, q, a.blocks, row_aligned) : one4;
            };
            fetch(k0 >> 4);
            w = s0 = s1 = one4;
            for (int q = k0 >> 2, first = q; q <= (k1 - 1) >> 2; ++q, ++groups) {
                const uint32_t g = groups & 1;
                if (q == first || (q & 3) == 0) {
                    w = next_w;
                    s0 = next0;
                    s1 = next1;
                    if (16 * ((q >> 2) + 1) < k1)
                        fetch((q >> 2) + 1);
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
                if (lane == 0) {
                    if (CG == 1)
                        mbar_arrive(&scale_full[g]);
                    else
                        arrive_cluster(in_cta(&scale_full[g], 0));
                }
            }
        }
        for (uint32_t i = groups > 2 ? groups - 2 : 0; i < groups; ++i)
            if (!wait(&scale_empty[i & 1], i >> 1 & 1, &guard))
                goto out;
    } else if (warp < kScaleWarp) {
        const uint32_t lanes = (uint32_t)warp << 21, chunk0 = smem_u32(stage0) + a.stages * a.stage_bytes;
        uint32_t done = 0, chunks = 0;
        for (int u = (int)cluster_index(); u < units; u += step, ++done) {
            const Tile t = tile_of(a, u);
            const uint32_t buf = done % kBuffers, acc = tmem + buf * a.tile + lanes;
            const int m = warp * 32 + lane, n = t.out * own_rows + (CG == 2 ? (int)rank * kRowsM : 0) + m, r0 = t.row * a.tile;
            const int used = min(a.tile, a.rows - r0);
            if (barrier_or<128>(2, !wait<true>(&acc_full[buf], done / kBuffers & 1, &guard)))
                goto out;
            tc_after();
            if (a.tma_out) {
                for (int c = 0; c < used; c += kChunk, ++chunks) {
                    float v[32];
                    tmem_load_pairs(acc + c, v);
                    tmem_load_pairs(acc + (16u << 16) + c, v + 16);
                    const uint32_t at = chunk0 + (chunks & 1) * kChunkBytes;
                    if (threadIdx.x == 0)
                        store_wait_read<1>();  // of this thread's two copies in flight the older one has left its buffer
                    named_barrier<128>(2);
                    tmem_wait<32>(v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // matrix j of the four: weight rows 8 j to 8 j + 7 of the warp's, activations' rows 8 i to 8 i + 7
                        const int row = 8 * i + (lane & 7), piece = (warp & 1) * 4 + lane / 8;
                        store_transposed(at + warp / 2 * (kChunkBytes / 2) + row * 128 + ((piece ^ (row & 7)) << 4),
                                         pack(v[4 * i], v[4 * i + 1]), pack(v[4 * i + 2], v[4 * i + 3]),
                                         pack(v[16 + 4 * i], v[17 + 4 * i]), pack(v[18 + 4 * i], v[19 + 4 * i]));
                    }
                    proxy_fence();
                    named_barrier<128>(2);
                    if (threadIdx.x == 0) {
                        // boxes of 64 outputs and 16 rows, those that begin inside the tile and the output
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const int from = n - m + 64 * (h / 2), row = c + 16 * (h & 1);
                            if (from < a.outs && row < used)
                                tma_store(&omap, at + h * (kChunkBytes / 4), from, r0 + row);
                        }
                        store_commit();
                    }
                }
            } else {
                for (int c = 0; c < used; c += 16) {
                    float v[16];
                    TmemLoad<16>::go(acc + c, v);
                    tmem_wait<16>(v);
                    if (CG == 1 && a.splits > 1) {
                        // the copies into the stages have all been used by now
                        float *const sums = (float *)stage0 + m;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            sums[(c + i) * kRowsM] = v[i];
                    } else if (n < a.outs) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c + i < used)
                                put(a, r0 + c + i, n, v[i]);
                    }
                }
            }
            tc_before();
            __syncwarp();
            if (lane == 0 && CG == 2)
                arrive_cluster(in_cta(&acc_empty[buf], 0));
        }
    }
out:
    if (threadIdx.x == 0)
        store_wait_read<0>();  // the buffers are the CTA's for as long as copies read them
    __syncwarp();
    if (CG == 1 && a.splits > 1) {
        cluster_sync();
        // each CTA adds its share of the tile's rows, rank by rank
        const Tile t = tile_of(a, (int)cluster_index());
        const int m = threadIdx.x % kRowsM, n = t.out * kRowsM + m, r0 = t.row * a.tile, used = min(a.tile, a.rows - r0);
        const int c1 = used * ((int)rank + 1) / a.splits;
        if (n < a.outs && threadIdx.x < 2 * kRowsM) {
            for (int c = used * (int)rank / a.splits + (int)threadIdx.x / kRowsM; c < c1; c += 2) {
                float v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    v[r] = r < a.splits ? load_cluster(in_cta((float *)stage0 + c * kRowsM + m, r)) : 0.0f;
                float sum = v[0];
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    sum += v[r];  // what is not there is 0
                put(a, r0 + c, n, sum);
            }
        }
    }
    __syncthreads();
    if (guard.dead) {
        // What is in flight lands before the memory is given back.  No barrier tells of all copies (a stage that only
        // one CTA of a pair filled never completes its phase), so a time is waited out that a copy takes many times over.
        if (warp == kIssueWarp && lead) {
            if (elected()) {
                Pair<CG>::commit(&landed);
                land(&landed, 0);
            }
        } else if (warp == kCopyWarp && lane == 0) {
            const long long since = clock64();
            while (clock64() - since < (1 << 22))
                ;
        }
        if (threadIdx.x == 0)
            report(a.status, SPEC_STATUS_INTERNAL);
        __syncwarp();
    }
    tc_before();
    if (linked)
        cluster_sync();
    else
        __syncthreads();
    tc_after();
    if (warp == kCopyWarp)
        Pair<CG>::dealloc(tmem, a.columns);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
struct Plan {
    bool pair;
    int tile, splits;
};

Plan plan(int rows, int outs, int blocks, int sms)
{
    const int out_tiles = (outs + kRowsM - 1) / kRowsM;
    Plan p{};
    if (rows > 64 && out_tiles >= 2 && (int64_t)rows * out_tiles > 128 * 76) {
        p.pair = true;
        p.splits = 1;
        const int pairs = (out_tiles + 1) / 2, units = sms / 2;
        int64_t best = INT64_MAX;
        for (int tile = 32; tile <= 240; tile += 16) {
            // a block takes as long as its instructions' issue, then as its products and copies: measured at 64 to 240 rows
            const int64_t tiles = (int64_t)pairs * ((rows + tile - 1) / tile),
                          cost = (tiles + units - 1) / units * std::max(tile + 160, 270);
            if (cost <= best) {
                best = cost;
                p.tile = tile;
            }
        }
        return p;
    }
    const int row_tiles = (rows + 127) / 128;
    p.tile = ((rows + row_tiles - 1) / row_tiles + 15) / 16 * 16;
    p.splits = 1;
    while (p.splits < 8 && (int64_t)out_tiles * row_tiles * p.splits * 2 <= 2 * sms && blocks >= 4 * p.splits)
        p.splits *= 2;
    return p;
}

constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];

constexpr uint32_t kMostShared = 227 * 1024;
// Bytes for the stages.  A CTA of a pair holds all of tensor memory, so nothing else that waits for some may be on its
// SM, where two clusters could each hold what the other waits for: it takes all of shared memory.  Two CTAs of splits
// share an SM, 256 columns each; a third one must not fit.
constexpr uint32_t kPairShared = kMostShared - 4096, kSplitShared = 110 * 1024;

spec_status device_sms(int *sms)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return SPEC_ERR_CUDA;
    }
    if (dev < 0 || dev >= kMaxDevices)
        return SPEC_ERR_UNSUPPORTED;
    int v = g_sms[dev].load(std::memory_order_acquire);
    if (!v) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaFuncSetAttribute(product_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitShared) != cudaSuccess ||
            cudaFuncSetAttribute(product_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairShared) != cudaSuccess) {
            cudaGetLastError();
            return SPEC_ERR_CUDA;
        }
        g_sms[dev].store(v, std::memory_order_release);
    }
    *sms = v;
    return SPEC_OK;
}

// [element, row], rows `stride` bytes apart; a box is 128 bytes of `box_rows` rows.
spec_status make_map(CUtensorMapDataType type, int element, void *at, int64_t dim, int64_t rows, int64_t stride, int box_rows,
                     CUtensorMap *map)
{
    const EncodeTiled encode = encoder();
    if (!encode)
        return SPEC_ERR_CUDA;
    const cuuint64_t size[2] = {(cuuint64_t)dim, (cuuint64_t)rows}, step[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {128u / (cuuint32_t)element, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return encode(map, type, 2, at, size, step, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? SPEC_OK
               : SPEC_ERR_INVALID_ARG;
}
spec_status make_map(const spec_coded *c, int box_rows, CUtensorMap *map)
{
    return make_map(CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c->codes, c->dim, c->rows, c->stride, box_rows, map);
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
    int sms = 0;
    st = device_sms(&sms);
    if (st != SPEC_OK)
        return st;
    Args a{};
    a.row_scale = rows->scale;
    a.row_scale_stride = rows->scale_stride;
    a.weight_scale = weight->scale;
    a.weight_scale_stride = weight->scale_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.rows = rows->rows;
    a.outs = weight->rows;
    a.blocks = scale_blocks(rows->dim);
    const Plan p = plan(a.rows, a.outs, a.blocks, sms);
    const int cg = p.pair ? 2 : 1;
    a.tile = p.tile;
    a.splits = p.splits;
    a.row_tiles = (a.rows + p.tile - 1) / p.tile;
    a.out_tiles = (a.outs + cg * kRowsM - 1) / (cg * kRowsM);
    if ((int64_t)a.row_tiles * a.out_tiles * p.splits > INT_MAX)
        return SPEC_ERR_UNSUPPORTED;
    // Eight weight tiles side by side share the rows that pass through L2; as many as stay there (32 MB of them) where the
    // rows themselves do not, so that those pass once (16,376 x 4,096 to 6,144: 224 us with 8, 197 with all 24; 1,280 x
    // 4,096 to 128,256: 395 us with 8, 440 with 64).
    a.group = 8;
    if ((int64_t)a.rows * a.blocks > (16 << 20) / kScaleBlock)
        a.group = std::max(8, (int)std::min<int64_t>(a.out_tiles, (32 << 20) / ((int64_t)cg * kRowsM * kScaleBlock * a.blocks)));
    a.b_bytes = (uint32_t)(p.tile / cg) * kScaleBlock;
    a.stage_bytes = (p.pair ? Depth<2>::value : Depth<1>::value) * (kABytes + a.b_bytes);  // a multiple of 1,024: tiles are multiples of 16, of 32 for a pair
    const uint32_t shared = p.pair ? kPairShared : kSplitShared;
    a.tma_out = dtype == SPEC_BF16 && p.splits == 1 && ((uintptr_t)out & 15u) == 0 && (out_stride * 2 & 15) == 0;
    a.stages = (int)std::min<uint32_t>(kMaxStages, (shared - 1024 - (a.tma_out ? 2 * kChunkBytes : 0)) / a.stage_bytes);
    a.columns = p.pair ? 512 : 256;
    // as in the unscaled kinds, and: bytes of the scales at bits 4 and 29 (set for each block), scales of powers of two (bit 23)
    a.idesc = (uint32_t)(weight->code == SPEC_E5M2) << 7 | (uint32_t)(rows->code == SPEC_E5M2) << 10 | (uint32_t)(p.tile >> 3) << 17 |
              1u << 23 | (uint32_t)(cg * kRowsM >> 7) << 27;
    a.wide_out = dtype == SPEC_F32;
    a.wait_limit = wait_limit();
    a.status = status;
    CUtensorMap wmap, rmap, omap{};
    if ((st = make_map(weight, kRowsM, &wmap)) != SPEC_OK || (st = make_map(rows, p.tile / cg, &rmap)) != SPEC_OK ||
        (a.tma_out && (st = make_map(CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, a.outs, a.rows, out_stride * 2, 16, &omap)) != SPEC_OK))
        return st;
    const int units = a.row_tiles * a.out_tiles;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.pair ? 2 : p.splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.pair ? 2 * std::min(units, sms / 2) : units * p.splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = (cudaStream_t)stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {&a, &wmap, &rmap, &omap};
    if (cudaLaunchKernelExC(&cfg, p.pair ? (const void *)product_kernel<2> : (const void *)product_kernel<1>, args) != cudaSuccess) {
        cudaGetLastError();
        return SPEC_ERR_CUDA;
    }
    return SPEC_OK;
}
