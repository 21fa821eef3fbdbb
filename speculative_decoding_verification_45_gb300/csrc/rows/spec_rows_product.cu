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
__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
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
    static __device__ __forceinline__ void load(const CUtensorMap *map, void *dst, uint32_t bar, int k, int row)
    {
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                         smem_u32(dst)),
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
    static __device__ __forceinline__ void load(const CUtensorMap *map, void *dst, uint32_t bar, int k, int row)
    {
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, "
                     "%4}], [%2];" ::"r"(smem_u32(dst)),
                     "l"(map), "r"(bar), "r"(k), "r"(row)
                     : "memory");
    }
};

// mbar_wait for a whole warp: all of its lanes go on, or none does.
template <bool NOW = false> __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile Guard *guard)
{
    return __all_sync(0xffffffffu, mbar_wait<NOW>(bar, parity, guard));
}

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

// Exponent bytes of blocks 4 g to 4 g + 3 of one row; 1 behind the last block (no instruction names those).
__device__ __forceinline__ uint32_t scale_word(const uint8_t *p, int64_t at, int g, int blocks, bool whole)
{
    p += at + 4 * g;
    if (whole && 4 * g + 4 <= blocks)
        return __ldg((const uint32_t *)p);
    uint32_t w = 0x7f7f7f7fu;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (4 * g + i < blocks)
            w = (w & ~(0xffu << 8 * i)) | (uint32_t)__ldg(p + i) << 8 * i;
    return w;
}

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

__device__ __forceinline__ void put(const Args &a, int64_t row, int col, float v)
{
    if (a.wide_out)
        ((float *)a.out)[row * a.out_stride + col] = v;
    else
        ((__nv_bfloat16 *)a.out)[row * a.out_stride + col] = __float2bfloat16_rn(v);
}

// ---------------------------------------------------------------------------
// The kernel.  CG: CTAs that issue products together.
// ---------------------------------------------------------------------------
template <int CG> __global__ void __launch_bounds__(kThreads, CG == 1 ? 2 : 1)
product_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap rmap)
{
    extern __shared__ uint8_t dynamic[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], scale_full[2], scale_empty[2], acc_full[2], acc_empty[2], landed;
    __shared__ uint32_t tmem_at;
    __shared__ Guard guard;
    uint8_t *const stage0 = (uint8_t *)(((uintptr_t)dynamic + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool lead = CG == 1 || rank == 0;
    const bool linked = CG == 2 || a.splits > 1;
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

    if (warp == kCopyWarp) {
        uint32_t it = 0;
        for (int u = (int)cluster_index(); u < units; u += step) {
            const Tile t = tile_of(a, u);
            const int n0 = t.out * own_rows + (CG == 2 ? (int)rank * kRowsM : 0), r0 = t.row * a.tile + (CG == 2 ? (int)rank * (a.tile / 2) : 0);
            for (int b = k0; b < k1; ++b, ++it) {
                const uint32_t s = it % a.stages;
                if (!wait(&empty[s], (it / a.stages & 1) ^ 1, &guard))
                    goto out;
                if (elected()) {
                    uint8_t *const at = stage0 + s * a.stage_bytes;
                    const uint32_t bar = CG == 1 ? smem_u32(&full[s]) : in_cta(&full[s], 0);
                    if (lead)
                        mbar_expect(&full[s], CG * a.stage_bytes);
                    Pair<CG>::load(&wmap, at, bar, b * kScaleBlock, n0);
                    Pair<CG>::load(&rmap, at + kABytes, bar, b * kScaleBlock, r0);
                }
                __syncwarp();
            }
        }
        // every stage given back: no arrival is on its way to this CTA's barriers when it ends
        for (uint32_t i = it > (uint32_t)a.stages ? it - a.stages : 0; i < it; ++i)
            if (!wait(&empty[i % a.stages], i / a.stages & 1, &guard))
                goto out;
    } else if (warp == kIssueWarp && lead) {
        uint32_t it = 0, groups = 0, done = 0;
        for (int u = (int)cluster_index(); u < units; u += step, ++done) {
            const uint32_t buf = done % kBuffers, acc = tmem + buf * a.tile;
            if (!wait(&acc_empty[buf], (done / kBuffers & 1) ^ 1, &guard))
                goto out;
            for (int b = k0; b < k1; ++b, ++it) {
                const uint32_t s = it % a.stages, g = groups & 1;
                if (b == k0 || (b & 3) == 0)
                    if (!wait(&scale_full[g], groups >> 1 & 1, &guard))
                        goto out;
                if (!wait(&full[s], it / a.stages & 1, &guard))
                    goto out;
                tc_after();
                const bool last = (b & 3) == 3 || b == k1 - 1;
                if (elected()) {
                    const uint32_t at = smem_u32(stage0 + s * a.stage_bytes);
                    // K-major, 128-byte rows in groups of eight; 32 elements further on are 32 bytes
                    const uint64_t da = smem_desc(at, 16, 1024, 2), db = smem_desc(at + kABytes, 16, 1024, 2);
                    const uint32_t id = a.idesc | (uint32_t)(b & 3) << 4 | (uint32_t)(b & 3) << 29;
                    const uint32_t sa = scales + g * kScaleColumns;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        Pair<CG>::mma(acc, da + 2 * k, db + 2 * k, id, sa, sa + 4, b > k0 || k > 0);
                    Pair<CG>::commit(&empty[s]);
                    if (last)
                        Pair<CG>::commit(&scale_empty[g]);
                    if (b == k1 - 1)
                        Pair<CG>::commit(&acc_full[buf]);
                }
                __syncwarp();
                groups += last;
            }
        }
    } else if (warp >= kScaleWarp && warp < kScaleWarp + 4) {
        const uint32_t lanes = (uint32_t)(warp - kScaleWarp) << 21;  // 32 lanes of tensor memory each, at bit 16
        const bool row_whole = ((uintptr_t)a.row_scale & 3) == 0 && (a.row_scale_stride & 3) == 0;
        const bool weight_whole = ((uintptr_t)a.weight_scale & 3) == 0 && (a.weight_scale_stride & 3) == 0;
        uint32_t groups = 0;
        for (int u = (int)cluster_index(); u < units; u += step) {
            const Tile t = tile_of(a, u);
            const int wb = t.out * CG + (CG == 2 ? (int)rank : 0), r0 = t.row * a.tile;
            const bool has = (int64_t)wb * kRowsM < a.outs;
            for (int q = k0 >> 2; q <= (k1 - 1) >> 2; ++q, ++groups) {
                const uint32_t g = groups & 1;
                uint32_t w[8];
                const uint32_t one = has ? scale_word(a.weight_scale, wb * a.weight_scale_stride, q, a.blocks, weight_whole) : 0x7f7f7f7fu;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = r0 + 32 * i + lane;
                    w[i] = 0x7f7f7f7fu;
                    if (32 * i < a.tile && row < a.rows)
                        w[i] = scale_word(a.row_scale, row * a.row_scale_stride, q, a.blocks, row_whole);
                }
                if (!wait(&scale_empty[g], (groups >> 1 & 1) ^ 1, &guard))
                    goto out;
                tc_after();
                const uint32_t at = scales + g * kScaleColumns + lanes;
                const uint32_t same[4] = {one, one, one, one};
                tmem_store<4>(at, same);
                if (a.tile > 128)
                    tmem_store<8>(at + 4, w);
                else
                    tmem_store<4>(at + 4, w);
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
        const uint32_t lanes = (uint32_t)warp << 21;
        uint32_t done = 0;
        for (int u = (int)cluster_index(); u < units; u += step, ++done) {
            const Tile t = tile_of(a, u);
            const uint32_t buf = done % kBuffers, acc = tmem + buf * a.tile + lanes;
            const int m = warp * 32 + lane, n = t.out * own_rows + (CG == 2 ? (int)rank * kRowsM : 0) + m, r0 = t.row * a.tile;
            const int used = min(a.tile, a.rows - r0);
            if (!wait<true>(&acc_full[buf], done / kBuffers & 1, &guard))
                goto out;
            tc_after();
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
            tc_before();
            __syncwarp();
            if (lane == 0 && CG == 2)
                arrive_cluster(in_cta(&acc_empty[buf], 0));
        }
    }
out:
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
        for (int tile = 32; tile <= 224; tile += 32) {
            const int64_t tiles = (int64_t)pairs * ((rows + tile - 1) / tile), cost = (tiles + units - 1) / units * (tile + 16);
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
constexpr uint32_t kPairShared = kMostShared - 1024, kSplitShared = 111 * 1024;

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

// [element, row] over the codes; a box is `rows` rows of one block.
spec_status make_map(const spec_coded *c, int rows, CUtensorMap *map)
{
    const EncodeTiled encode = encoder();
    if (!encode)
        return SPEC_ERR_CUDA;
    const cuuint64_t size[2] = {(cuuint64_t)c->dim, (cuuint64_t)c->rows}, step[1] = {(cuuint64_t)c->stride};
    const cuuint32_t box[2] = {kScaleBlock, (cuuint32_t)rows}, one[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, c->codes, size, step, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? SPEC_OK
               : SPEC_ERR_INVALID_ARG;
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
    a.group = 8;
    a.b_bytes = (uint32_t)(p.tile / cg) * kScaleBlock;
    a.stage_bytes = kABytes + a.b_bytes;  // a multiple of 1,024: tiles are multiples of 16, of 32 for a pair
    const uint32_t shared = p.pair ? kPairShared : kSplitShared;
    a.stages = (int)std::min<uint32_t>(kMaxStages, (shared - 1024) / a.stage_bytes);
    a.columns = p.pair ? 512 : 256;
    // as in the unscaled kinds, and: bytes of the scales at bits 4 and 29 (set for each block), scales of powers of two (bit 23)
    a.idesc = (uint32_t)(weight->code == SPEC_E5M2) << 7 | (uint32_t)(rows->code == SPEC_E5M2) << 10 | (uint32_t)(p.tile >> 3) << 17 |
              1u << 23 | (uint32_t)(cg * kRowsM >> 7) << 27;
    a.wide_out = dtype == SPEC_F32;
    a.wait_limit = wait_limit();
    a.status = status;
    CUtensorMap wmap, rmap;
    if ((st = make_map(weight, kRowsM, &wmap)) != SPEC_OK || (st = make_map(rows, p.tile / cg, &rmap)) != SPEC_OK)
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
    void *args[] = {&a, &wmap, &rmap};
    if (cudaLaunchKernelExC(&cfg, p.pair ? (const void *)product_kernel<2> : (const void *)product_kernel<1>, args) != cudaSuccess) {
        cudaGetLastError();
        return SPEC_ERR_CUDA;
    }
    return SPEC_OK;
}
