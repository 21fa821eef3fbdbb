// spec_ptx.cuh -- barriers, copies and tensor memory of sm_103a as the kernels of
// csrc/cache and csrc/rows use them.
#ifndef SPEC_PTX_CUH
#define SPEC_PTX_CUH

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace specc {

// Host helpers (spec_cache_attend.cu).
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encoder();  // cuTensorMapEncodeTiled, or null
int wait_limit();       // clocks that a wait inside a kernel may take

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

}  // namespace specc

#endif
