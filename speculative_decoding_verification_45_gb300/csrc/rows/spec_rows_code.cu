// spec_rows_code.cu -- rows and weights to 8 bits: as they are (spec_rows_quantise),
// after the residual's addition and the root-mean-square norm (spec_rows_norm),
// and as the product of an activated gate and its partner (spec_rows_gate).
// include/spec_verify.h states the operations.
//
// Each is one pass over memory, which bounds it: an element is read once, kept in
// registers while its block's (or row's) largest is found, and written as a code.
// A thread takes eight neighbouring elements, so sixteen lanes hold a block of 128
// and agree on its scale by four shuffles.  All arithmetic is 32-bit; the only
// rounding to fewer bits is that to the code, and of the sum that spec_rows_norm
// writes back (which its norm does not read again: it takes the 32-bit sum).

#include <type_traits>

#include "../cache/spec_ptx.cuh"
#include "spec_rows.cuh"

using namespace specc;

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = kScaleBlock / 8;  // of a block

struct Eight {  // values, two by two for the instructions that take two
    float2 v[4];
};

__device__ __forceinline__ float2 unpack(uint32_t two) { return {__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u)}; }

// The largest magnitude's bits: magnitudes as integers are in the same order.  From 0x7f800000 up it stands for an infinity
// (or, in `most_of` 16-bit values, a NaN; the other form passes over those).
constexpr uint32_t kInfinity = 0x7f800000u;

__device__ __forceinline__ uint32_t most(const Eight &e)
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = fmaxf(fmaxf(m, fabsf(e.v[i].x)), fabsf(e.v[i].y));
    return __float_as_uint(m);
}

// Eight elements as they lie in memory.  lowest(): the bits of the one furthest below 0, which are larger than a positive
// number's as an integer's (a NaN's, with its sign set, are larger still).
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
    uint4 q;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { q = *(const uint4 *)p; }
    __device__ __forceinline__ void clear() { q = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ Eight values() const { return {{unpack(q.x), unpack(q.y), unpack(q.z), unpack(q.w)}}; }
    __device__ __forceinline__ uint32_t most_of() const
    {
        constexpr uint32_t kMagnitude = 0x7fff7fffu;
        const uint32_t m = max_halves(max_halves(q.x & kMagnitude, q.y & kMagnitude), max_halves(q.z & kMagnitude, q.w & kMagnitude));
        return max(m << 16, m & 0xffff0000u);
    }
    __device__ __forceinline__ uint32_t lowest() const
    {
        const uint32_t m = max_halves(max_halves(q.x, q.y), max_halves(q.z, q.w));
        return max(m << 16, m & 0xffff0000u);
    }
};
template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = *(const float4 *)p;
        b = *(const float4 *)(p + 4);
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0, 0, 0, 0); }
    __device__ __forceinline__ Eight values() const { return {{{a.x, a.y}, {a.z, a.w}, {b.x, b.y}, {b.z, b.w}}}; }
    __device__ __forceinline__ uint32_t most_of() const { return most(values()); }
    __device__ __forceinline__ uint32_t lowest() const
    {
        const auto of = [](const float4 &f) {
            return max(max(__float_as_uint(f.x), __float_as_uint(f.y)), max(__float_as_uint(f.z), __float_as_uint(f.w)));
        };
        return max(of(a), of(b));
    }
};

__device__ __forceinline__ uint32_t pack(float2 a)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
    return *(const uint32_t *)&h;
}
__device__ __forceinline__ void store(__nv_bfloat16 *p, const Eight &e)
{
    *(uint4 *)p = make_uint4(pack(e.v[0]), pack(e.v[1]), pack(e.v[2]), pack(e.v[3]));
}
__device__ __forceinline__ void store(float *p, const Eight &e)
{
    *(float4 *)p = make_float4(e.v[0].x, e.v[0].y, e.v[1].x, e.v[1].y);
    *(float4 *)(p + 4) = make_float4(e.v[2].x, e.v[2].y, e.v[3].x, e.v[3].y);
}

// The largest finite magnitude's bits, for the rare block that holds something else.
__device__ __forceinline__ uint32_t most_finite(const Eight &e)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(i & 1 ? e.v[i / 2].y : e.v[i / 2].x) & 0x7fffffffu;
        m = max(m, u < kInfinity ? u : 0u);
    }
    return m;
}
// Over the sixteen lanes of a block.
__device__ __forceinline__ uint32_t of_block(uint32_t m)
{
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1)
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// The scale's exponent byte, from the largest magnitude's bits.
__device__ __forceinline__ uint32_t exponent_byte(uint32_t most, int code)
{
    return __float_as_uint(scale_for(__uint_as_float(most), code)) >> 23;
}

// Codes of eight elements; the byte is in [27, 247], so the reciprocal is a normal power of two.  finite: no infinity is
// among them (it would become the largest code; a NaN is the code NaN either way).
__device__ __forceinline__ uint2 encode(const Eight &e, uint32_t byte, int code, bool finite)
{
    const float inv = __uint_as_float((254u - byte) << 23);
    uint32_t h[4];
    float2 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = mul2(e.v[i], {inv, inv});
    if (!finite) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = encode2(x[i].x, x[i].y, code);
    } else if (code == SPEC_E4M3) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = encode2_finite(x[i].x, x[i].y, SPEC_E4M3);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = encode2_finite(x[i].x, x[i].y, SPEC_E5M2);
    }
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

// The scale's byte for the sixteen lanes of a block, from each lane's largest magnitude; whether all in the warp is finite.
__device__ __forceinline__ uint32_t block_byte(uint32_t m, const Eight &e, int code, bool *finite)
{
    m = of_block(m);
    *finite = !__any_sync(0xffffffffu, m >= kInfinity);
    if (!*finite)
        m = of_block(most_finite(e));
    return exponent_byte(m, code);
}

struct Out {
    uint8_t *codes, *scale;
    int64_t stride, scale_stride;
    int rows, dim, code;
};

// ---------------------------------------------------------------------------
// One scale for each row and 128 elements
// ---------------------------------------------------------------------------
struct Plain {
    static constexpr int kInputs = 1;
};
// a / (1 + exp(-z)) * b.  exp by the fast base-2 form, off by 2^-22; its argument goes through up to four roundings and is off
// by 2^-22 of itself, which is the result's error where z is negative (where it is positive the sum is next to 1).
template <bool GELU> struct Gated {
    static constexpr int kInputs = 2;
    // Above this exp(-z) is below 2^125 and the sum's reciprocal a normal number.  Further down the result would be 0, which with
    // a large b it is not: such gates are looked for in the inputs' bits, and eight with one among them go a way of their own.
    // (4,094 x 16,384 in bf16: 54 us, 52.6 without that way, 60 if z is what is looked at, which holds more registers.)
    static constexpr float kLow = GELU ? -9.875f : -86.0f;
    static __device__ __forceinline__ float2 exponent(float2 g)  // -z in units of log 2
    {
        // 0.5 (1 + tanh(y)) = 1 / (1 + exp(-2 y)), y = sqrt(2 / pi) (g + 0.044715 g^3); exp(x) = 2^(x log2 e)
        constexpr float kLog2e = 1.44269504088896f, kOne = -1.59576912160573f * kLog2e, kThree = -0.0713548162726003f * kLog2e;
        if (GELU)
            return mul2(g, fma2(mul2(g, {kThree, kThree}), g, {kOne, kOne}));
        return mul2(g, {-kLog2e, -kLog2e});
    }
    static __device__ __forceinline__ float2 product(float2 g, float2 z, float2 b)
    {
        const float2 d = add2({exp2_fast(z.x), exp2_fast(z.y)}, {1.0f, 1.0f});
        float2 s;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(d.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(d.y));
        return mul2(mul2(g, s), b);
    }
    // Past 2^125 the exponential is the sum, and its four roots divide by turns.
    static __device__ __forceinline__ float far_below(float g, float z, float b)
    {
        const float root = exp2_fast(-0.25f * z);
        return b * root * root * root * (g * root);
    }
    template <typename Raw> static __device__ __forceinline__ Eight of(const Raw &a, const Raw &b)
    {
        const Eight g = a.values(), u = b.values();
        Eight r;
        if (a.lowest() < __float_as_uint(kLow)) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r.v[i] = product(g.v[i], exponent(g.v[i]), u.v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 z = exponent(g.v[i]);
                r.v[i] = product(g.v[i], z, u.v[i]);
                if (z.x > 125.0f)
                    r.v[i].x = far_below(g.v[i].x, z.x, u.v[i].x);
                if (z.y > 125.0f)
                    r.v[i].y = far_below(g.v[i].y, z.y, u.v[i].y);
            }
        }
        return r;
    }
};

struct Inputs {
    const void *a, *b;
    int64_t a_stride, b_stride;
};

// Chunks of eight in order: slots of a row are filled up to whole blocks, so that the sixteen lanes
// of a block are neighbours.  per_slots: ceil(2^32 / slots), exact for what is divided by it (below slots + 512).
constexpr int kUnroll = 2;

template <typename T, typename F> __global__ void __launch_bounds__(kThreads) code_kernel(const Inputs in, const Out o,
                                                                                         const int slots, const uint32_t per_slots)
{
    // in units of a block's lanes the first chunk's place fits 32 bits
    const uint32_t blocks = (uint32_t)slots / kLanes, first = blockIdx.x * (kThreads * kUnroll / kLanes), above = first / blocks;
    const int64_t row0 = above;
    const uint32_t slot0 = (first - above * blocks) * kLanes + threadIdx.x;
    after_previous();
    Raw<T> a[kUnroll], b[kUnroll];
    int64_t row[kUnroll];
    int col[kUnroll];
    bool in_row[kUnroll], in_all[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint32_t s = slot0 + u * kThreads, down = __umulhi(s, per_slots);
        row[u] = row0 + down;
        col[u] = (int)(s - down * (uint32_t)slots) * 8;
        in_all[u] = row[u] < o.rows;
        in_row[u] = in_all[u] && col[u] < o.dim;
        a[u].clear();
        b[u].clear();
        if (in_row[u]) {
            a[u].load((const T *)in.a + row[u] * in.a_stride + col[u]);
            if (F::kInputs == 2)
                b[u].load((const T *)in.b + row[u] * in.b_stride + col[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        Eight e;
        uint32_t m;
        if constexpr (F::kInputs == 2) {
            e = F::of(a[u], b[u]);
            m = most(e);
        } else {
            e = a[u].values();
            m = a[u].most_of();
        }
        bool finite;
        const uint32_t byte = block_byte(m, e, o.code, &finite);
        if (in_row[u])
            *(uint2 *)(o.codes + row[u] * o.stride + col[u]) = encode(e, byte, o.code, finite);
        if (in_all[u] && (threadIdx.x & (kLanes - 1)) == 0)
            o.scale[row[u] * o.scale_stride + col[u] / kScaleBlock] = (uint8_t)byte;
    }
}

// ---------------------------------------------------------------------------
// One scale for each 128 x 128: a CTA a block, which stays in registers as it was read
// ---------------------------------------------------------------------------
constexpr int kBlockThreads = 512;

// Three CTAs to an SM leave the registers that a block in bf16 takes, two those of one in fp32, which spilled with three
// (32,000 x 4,096: 60.0 us in bf16; in fp32 95.6, 111.4 with three).
template <typename T> __global__ void __launch_bounds__(kBlockThreads, sizeof(T) == 2 ? 3 : 2) block_kernel(const T *x, int64_t x_stride, const Out o)
{
    constexpr int kEach = kScaleBlock * kLanes / kBlockThreads;
    __shared__ uint32_t found[kBlockThreads / 32];
    const int col = blockIdx.x * kScaleBlock + (threadIdx.x & (kLanes - 1)) * 8;
    const int64_t row0 = (int64_t)blockIdx.y * kScaleBlock + threadIdx.x / kLanes;
    after_previous();
    Raw<T> raw[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t row = row0 + i * (kBlockThreads / kLanes);
        raw[i].clear();
        if (row < o.rows && col < o.dim)
            raw[i].load(x + row * x_stride + col);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        m = max(m, raw[i].most_of());
    const bool finite = !__syncthreads_or(m >= kInfinity);
    if (!finite) {
        m = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            m = max(m, most_finite(raw[i].values()));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0)
        found[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBlockThreads / 32; ++i)
        m = max(m, found[i]);
    const uint32_t byte = exponent_byte(m, o.code);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t row = row0 + i * (kBlockThreads / kLanes);
        if (row < o.rows && col < o.dim)
            *(uint2 *)(o.codes + row * o.stride + col) = encode(raw[i].values(), byte, o.code, finite);
    }
    if (threadIdx.x == 0)
        o.scale[(int64_t)blockIdx.y * o.scale_stride + blockIdx.x] = (uint8_t)byte;
}

// ---------------------------------------------------------------------------
// Residual, norm, codes: a CTA a row, or a warp for up to 1,024 elements, which stays in registers
// ---------------------------------------------------------------------------
struct NormArgs {
    const void *x, *residual, *weight;
    void *sum;
    int64_t x_stride, residual_stride, sum_stride;
    float eps;
    int weight_bf16;
};

struct None {};  // no residual

// EACH: chunks of eight to a thread.  WARP: eight rows to a CTA, so that short ones do not each cost a CTA's start
// (16,376 of 512 elements: 17.4 us with a CTA each, 9.9 so).  EARLY: the weight is read beside the row, not when the row's
// sum is known, for which more of the row's registers are in use at once (`launch_norm` has the rule).
template <typename T, typename R, int EACH, bool WARP, bool EARLY> __global__ void __launch_bounds__(WARP ? kThreads : 512)
norm_kernel(const NormArgs a, const Out o)
{
    constexpr bool kResidual = !std::is_same<R, None>::value;
    using S = typename std::conditional<kResidual, R, float>::type;
    __shared__ float part[32];
    const int threads = WARP ? 32 : blockDim.x, mine = WARP ? threadIdx.x & 31 : threadIdx.x;  // of the row
    const int64_t row = WARP ? (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32 : blockIdx.x;
    after_previous();
    if (WARP && row >= o.rows)
        return;
    Raw<T> x[EACH];
    Raw<S> r[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int col = (i * threads + mine) * 8;
        x[i].clear();
        r[i].clear();
        if (col < o.dim) {
            x[i].load((const T *)a.x + row * a.x_stride + col);
            if (kResidual)
                r[i].load((const S *)a.residual + row * a.residual_stride + col);
        }
    }
    const auto weight_at = [&](int col) {
        Eight w{{{1, 1}, {1, 1}, {1, 1}, {1, 1}}};
        if (a.weight && col < o.dim) {
            if (a.weight_bf16) {
                Raw<__nv_bfloat16> raw;
                raw.load((const __nv_bfloat16 *)a.weight + col);
                w = raw.values();
            } else {
                Raw<float> raw;
                raw.load((const float *)a.weight + col);
                w = raw.values();
            }
        }
        return w;
    };
    Eight early[EARLY ? EACH : 1];
    if (EARLY)
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            early[EARLY ? i : 0] = weight_at((i * threads + mine) * 8);
    Eight h[EACH];
    float2 two = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int col = (i * threads + mine) * 8;
        h[i] = x[i].values();
        if (kResidual) {
            const Eight more = r[i].values();
#pragma unroll
            for (int j = 0; j < 4; ++j)
                h[i].v[j] = add2(h[i].v[j], more.v[j]);
            if (col < o.dim)
                store((S *)a.sum + row * a.sum_stride + col, h[i]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            two = fma2(h[i].v[j], h[i].v[j], two);
    }
    // of the row, from each thread's share
    const auto sum_of = [&](float2 share) {
        float sum = share.x + share.y;
#pragma unroll
        for (int k = 16; k; k >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, k);
        if (!WARP) {
            if ((threadIdx.x & 31) == 0)
                part[threadIdx.x / 32] = sum;
            __syncthreads();
            sum = (threadIdx.x & 31) < blockDim.x / 32 ? part[threadIdx.x & 31] : 0.0f;
#pragma unroll
            for (int k = 16; k; k >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, k);
        }
        return sum;
    };
    const float squares = sum_of(two);
    float factor = __frsqrt_rn(__fdiv_rn(squares, (float)o.dim) + a.eps);
    if (__float_as_uint(squares) >= kInfinity) {
        // The squares pass 32 bits, at elements of 2^64 / sqrt(dim) already, where the row may yet be finite: those of 2^-72 of
        // it stay below 2^(112 + 15).  The factor is 2^-128 at least, where 32 bits hold 21 digits of it.
        constexpr float kDown = 0x1p-72f;
        two = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < EACH; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = mul2(h[i].v[j], {kDown, kDown});
                two = fma2(v, v, two);
            }
        if (!WARP)
            __syncthreads();
        factor = __frsqrt_rn(__fdiv_rn(sum_of(two), (float)o.dim) + a.eps * kDown * kDown) * kDown;
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int slot = i * threads + mine, col = slot * 8;
        const Eight w = EARLY ? early[EARLY ? i : 0] : weight_at(col);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h[i].v[j] = mul2(mul2(h[i].v[j], {factor, factor}), w.v[j]);
        bool finite;
        const uint32_t byte = block_byte(most(h[i]), h[i], o.code, &finite);
        if (col < o.dim) {
            *(uint2 *)(o.codes + row * o.stride + col) = encode(h[i], byte, o.code, finite);
            if ((mine & (kLanes - 1)) == 0)
                o.scale[row * o.scale_stride + slot / kLanes] = (uint8_t)byte;
        }
    }
}

Out make_out(const spec_coded *c)
{
    return {(uint8_t *)c->codes, c->scale, c->stride, c->scale_stride, c->rows, c->dim, c->code};
}

template <typename T, typename F> spec_status launch_code(const Inputs &in, const spec_coded *out, cudaStream_t stream)
{
    const int slots = scale_blocks(out->dim) * kLanes;
    const int64_t all = (int64_t)out->rows * slots, each = kThreads * kUnroll, ctas = (all + each - 1) / each;
    if (all / kLanes > INT_MAX)
        return SPEC_ERR_UNSUPPORTED;
    const uint32_t per = (uint32_t)(((1ull << 32) + slots - 1) / slots);
    return launch(code_kernel<T, F>, dim3((unsigned)ctas), kThreads, 0, 1, stream, in, make_out(out), slots, per);
}

template <typename T, typename R, int EACH, bool WARP>
spec_status launch_norm(bool early, unsigned ctas, int threads, cudaStream_t stream, const NormArgs &a, const Out &o)
{
    if (early)
        return launch(norm_kernel<T, R, EACH, WARP, EACH <= 4>, dim3(ctas), threads, 0, 1, stream, a, o);
    return launch(norm_kernel<T, R, EACH, WARP, false>, dim3(ctas), threads, 0, 1, stream, a, o);
}

template <typename T, typename R> spec_status launch_norm(const NormArgs &a, const spec_coded *out, cudaStream_t stream)
{
    const int slots = scale_blocks(out->dim) * kLanes;
    const Out o = make_out(out);
    // The weight is read early where all rows are at work at once, 16,384 elements to each of 152 SMs, and only latency
    // counts (1 x 4,096: 3.2 to 2.3 us; 1 x 8,192: 4.9 to 3.0; 304 x 8,192: 6.0 to 5.0).  With more, its registers cost rows
    // in flight (608 x 8,192: 8.1 us late, 9.3 early; 16,376: 136 and 178).
    const bool early = (int64_t)out->rows * out->dim <= 152 * 16384;
    const unsigned rows = (unsigned)out->rows, few = (rows + kThreads / 32 - 1) / (kThreads / 32);
    if (slots <= 32)
        return launch_norm<T, R, 1, true>(early, few, kThreads, stream, a, o);
    if (slots <= 64)
        return launch_norm<T, R, 2, true>(early, few, kThreads, stream, a, o);
    if (slots <= 128)
        return launch_norm<T, R, 4, true>(early, few, kThreads, stream, a, o);
    const auto threads = [&](int each) { return ((slots + each - 1) / each + 31) / 32 * 32; };
    if (slots <= 512)
        return launch_norm<T, R, 2, false>(early, rows, threads(2), stream, a, o);
    if (slots <= 2048)
        return launch_norm<T, R, 4, false>(early, rows, threads(4), stream, a, o);
    return launch_norm<T, R, 8, false>(early, rows, threads(8), stream, a, o);
}

template <typename T> spec_status norm_of(const NormArgs &a, int residual, const spec_coded *out, cudaStream_t stream)
{
    if (!a.residual)
        return launch_norm<T, None>(a, out, stream);
    return residual == SPEC_BF16 ? launch_norm<T, __nv_bfloat16>(a, out, stream) : launch_norm<T, float>(a, out, stream);
}

}  // namespace

extern "C" {

spec_status spec_rows_quantise(const void *x, int64_t x_stride, spec_dtype dtype, const spec_coded *out, int block_rows,
                               void *stream)
{
    NvtxScope nvtx("spec_rows_quantise");
    const spec_status st = check_coded(out);
    if (st != SPEC_OK)
        return st;
    if (bad_dtype(dtype) || (block_rows != 1 && block_rows != kScaleBlock))
        return SPEC_ERR_UNSUPPORTED;
    if (out->rows == 0)
        return SPEC_OK;
    if (bad_rows(x, x_stride, dtype))
        return SPEC_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    if (block_rows == 1) {
        const Inputs in{x, nullptr, x_stride, 0};
        return dtype == SPEC_BF16 ? launch_code<__nv_bfloat16, Plain>(in, out, s) : launch_code<float, Plain>(in, out, s);
    }
    const int64_t down = ((int64_t)out->rows + kScaleBlock - 1) / kScaleBlock;
    if (down > 65535)
        return SPEC_ERR_UNSUPPORTED;
    const dim3 grid(scale_blocks(out->dim), (unsigned)down);
    return dtype == SPEC_BF16 ? launch(block_kernel<__nv_bfloat16>, grid, kBlockThreads, 0, 1, s, (const __nv_bfloat16 *)x, x_stride, make_out(out))
                              : launch(block_kernel<float>, grid, kBlockThreads, 0, 1, s, (const float *)x, x_stride, make_out(out));
}

spec_status spec_rows_norm(const void *x, int64_t x_stride, spec_dtype dtype, const void *residual,
                           int64_t residual_stride, spec_dtype residual_dtype, const void *weight,
                           spec_dtype weight_dtype, float eps, void *sum, int64_t sum_stride, const spec_coded *out,
                           void *stream)
{
    NvtxScope nvtx("spec_rows_norm");
    const spec_status st = check_coded(out);
    if (st != SPEC_OK)
        return st;
    if (bad_dtype(dtype) || (residual && bad_dtype(residual_dtype)) || (weight && bad_dtype(weight_dtype)) ||
        out->dim > SPEC_MAX_NORM_ROW)
        return SPEC_ERR_UNSUPPORTED;
    if (!(eps >= 0x1p-126f) || !(eps - eps == 0.0f))
        return SPEC_ERR_INVALID_ARG;
    if (out->rows == 0)
        return SPEC_OK;
    if (bad_rows(x, x_stride, dtype) || ((uintptr_t)weight & 15u) || !residual != !sum ||
        (residual && (bad_rows(residual, residual_stride, residual_dtype) || bad_rows(sum, sum_stride, residual_dtype) ||
                      sum_stride < out->dim)))
        return SPEC_ERR_INVALID_ARG;
    const NormArgs a{x, residual, weight, sum, x_stride, residual_stride, sum_stride, eps, weight_dtype == SPEC_BF16};
    return dtype == SPEC_BF16 ? norm_of<__nv_bfloat16>(a, residual_dtype, out, (cudaStream_t)stream)
                              : norm_of<float>(a, residual_dtype, out, (cudaStream_t)stream);
}

spec_status spec_rows_gate(const void *gate, int64_t gate_stride, const void *up, int64_t up_stride, spec_dtype dtype,
                           spec_act act, const spec_coded *out, void *stream)
{
    NvtxScope nvtx("spec_rows_gate");
    const spec_status st = check_coded(out);
    if (st != SPEC_OK)
        return st;
    if (bad_dtype(dtype) || (act != SPEC_SILU && act != SPEC_GELU_TANH))
        return SPEC_ERR_UNSUPPORTED;
    if (out->rows == 0)
        return SPEC_OK;
    if (bad_rows(gate, gate_stride, dtype) || bad_rows(up, up_stride, dtype))
        return SPEC_ERR_INVALID_ARG;
    const Inputs in{gate, up, gate_stride, up_stride};
    const cudaStream_t s = (cudaStream_t)stream;
    if (dtype == SPEC_BF16)
        return act == SPEC_SILU ? launch_code<__nv_bfloat16, Gated<false>>(in, out, s)
                                : launch_code<__nv_bfloat16, Gated<true>>(in, out, s);
    return act == SPEC_SILU ? launch_code<float, Gated<false>>(in, out, s) : launch_code<float, Gated<true>>(in, out, s);
}

}  // extern "C"
