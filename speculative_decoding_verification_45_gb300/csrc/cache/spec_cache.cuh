// spec_cache.cuh -- what the kernels of the 8-bit key/value cache share
// (include/spec_verify.h states the operations).
#ifndef SPEC_CACHE_CUH
#define SPEC_CACHE_CUH

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <climits>
#include <cstdint>

#include "spec_verify.h"

namespace specc {

constexpr int kMaxBlock = 128;

// Largest code of each form: 1.75 * 2^8 and 1.75 * 2^15.
__device__ __forceinline__ int code_top_exponent(int code) { return code == SPEC_E4M3 ? 8 : 15; }

// The smallest power of two s with amax <= s * 1.75 * 2^top, and at least 2^-100, from the bits
// of amax (finite, >= 0): amax = f * 2^e with f in [1, 2) needs 2^(e - top), twice that for f > 1.75.
__device__ __forceinline__ float scale_for(float amax, int code)
{
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - code_top_exponent(code) + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    // subnormal amax has e = -127 - top or one more: under the floor either way
    return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}

__device__ __forceinline__ bool is_pow2(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0; }

// x / s rounded once; exact for a power of two, whose reciprocal is one too.
struct Divider {
    float inv, s;
    bool exact;
    __device__ explicit Divider(float scale) : inv(1.0f / scale), s(scale), exact(is_pow2(scale)) {}
    __device__ __forceinline__ float operator()(float x) const { return exact ? x * inv : __fdiv_rn(x, s); }
};

__device__ __forceinline__ float2 decode2(uint16_t two, int code)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(two, code == SPEC_E4M3 ? __NV_E4M3 : __NV_E5M2);
    return __half22float2(__half2(h));
}

// Two finite values to codes, nearest even.
__device__ __forceinline__ uint16_t encode2_finite(float a, float b, int code)
{
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, code == SPEC_E4M3 ? __NV_E4M3 : __NV_E5M2);
}

// Two values to codes; a value that is not finite becomes NaN.
__device__ __forceinline__ uint16_t encode2(float a, float b, int code)
{
    return encode2_finite(isfinite(a) ? a : __int_as_float(0x7fffffff), isfinite(b) ? b : __int_as_float(0x7fffffff), code);
}

__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b)  // of unsigned 16-bit halves
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Codes times f <= 1, to codes.  A power of two that 16-bit floats hold (2^-24 is
// their smallest) is multiplied in them: a product that they do not hold exactly
// is below half the smallest code.
struct Mover {
    float f;
    __half2 f2;
    bool halves;
    __device__ explicit Mover(float factor)
        : f(factor), f2(__float2half2_rn(factor)), halves(is_pow2(factor) && factor >= 0x1p-24f)
    {
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t x, int code) const  // four of them
    {
        // an infinity (e5m2) takes the other way, where it becomes NaN
        if (halves && !(code == SPEC_E5M2 && __vcmpeq4(x & 0x7f7f7f7fu, 0x7c7c7c7cu))) {
            const __nv_fp8_interpretation_t kind = code == SPEC_E4M3 ? __NV_E4M3 : __NV_E5M2;
            const __half2 lo = __hmul2(__half2(__nv_cvt_fp8x2_to_halfraw2((uint16_t)x, kind)), f2),
                          hi = __hmul2(__half2(__nv_cvt_fp8x2_to_halfraw2((uint16_t)(x >> 16), kind)), f2);
            return (uint32_t)__nv_cvt_halfraw2_to_fp8x2(__half2_raw(lo), __NV_SATFINITE, kind) |
                   (uint32_t)__nv_cvt_halfraw2_to_fp8x2(__half2_raw(hi), __NV_SATFINITE, kind) << 16;
        }
        const float2 lo = decode2((uint16_t)x, code), hi = decode2((uint16_t)(x >> 16), code);
        return (uint32_t)encode2(lo.x * f, lo.y * f, code) | (uint32_t)encode2(hi.x * f, hi.y * f, code) << 16;
    }
};

// One sequence's lengths, checked: `len` cached tokens (0 where they are invalid).
struct Seq {
    int len, m;  // tokens, new ones
    bool ok;
};

__device__ __forceinline__ Seq sequence(const spec_cache &c, const int32_t *lengths, const int32_t *num_new, int n,
                                        int b, bool after)
{
    const long long room = (long long)c.max_blocks * c.block;
    const int len = lengths[b], m = num_new ? num_new[b] : n;
    Seq s{len, m, true};
    // after: the new tokens are among the `len`; else they follow them
    s.ok = len >= 0 && m >= 0 && m <= n && (after ? len <= room && m <= len : (long long)len + m <= room);
    if (!s.ok)
        s.len = s.m = 0;
    return s;
}

__device__ __forceinline__ int page_of(const spec_cache &c, int b, int block)
{
    const int p = c.block_table[(size_t)b * c.table_stride + block];
    return (unsigned)p < (unsigned)c.num_pages ? p : -1;
}

__device__ __forceinline__ void report(uint32_t *status, uint32_t bit)
{
    if (status)
        atomicOr(status, bit);
}

struct NvtxScope {
    explicit NvtxScope(const char *name) { nvtxRangePushA(name); }
    ~NvtxScope() { nvtxRangePop(); }
};

inline bool bad4(const void *p, bool required) { return (required && !p) || ((uintptr_t)p & 3u); }

// Host checks that every entry point makes of the cache's description.
inline spec_status check_cache(const spec_cache *c)
{
    if (!c || c->batch < 0 || c->batch > SPEC_MAX_BATCH || c->max_blocks < 1 || c->num_pages < 1 ||
        c->kv_heads < 1 || c->table_stride < c->max_blocks)
        return SPEC_ERR_INVALID_ARG;
    if ((c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) ||
        (c->dim != 64 && c->dim != 128) || (c->code != SPEC_E4M3 && c->code != SPEC_E5M2))
        return SPEC_ERR_UNSUPPORTED;
    if ((int64_t)c->max_blocks * c->block > SPEC_MAX_CACHED)
        return SPEC_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
        if (c->k_stride[i] < 16 || c->v_stride[i] < 16 || (c->k_stride[i] & 15) || (c->v_stride[i] & 15) ||
            c->k_stride[i] >= (1ll << 40) || c->v_stride[i] >= (1ll << 40))
            return SPEC_ERR_INVALID_ARG;
    const void *p16[] = {c->k, c->v};
    for (const void *p : p16)
        if (!p || ((uintptr_t)p & 15u))
            return SPEC_ERR_INVALID_ARG;
    if (bad4(c->k_scale, true) || bad4(c->v_scale, true) || bad4(c->block_table, c->batch > 0) ||
        ((uintptr_t)c->positions & 15u))
        return SPEC_ERR_INVALID_ARG;
    return SPEC_OK;
}

inline spec_status launched()
{
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace specc

#endif
