// spec_cache_attend.cu -- host side of attention over the 8-bit key/value cache
// and of the weights that its tokens received (spec_cache_attend,
// spec_cache_weigh): argument checks, the launch, the tensor maps.  The kernels
// are in spec_cache_attend.cuh.

#include <atomic>

#include "spec_cache_attend.cuh"

using namespace specc;

namespace {

std::atomic<int> g_wait_limit{INT_MAX};  // clocks

}  // namespace

int specc::wait_limit() { return g_wait_limit.load(std::memory_order_relaxed); }

EncodeTiled specc::encoder()
{
    static const EncodeTiled f = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return (EncodeTiled)p;
    }();
    return f;
}

namespace {

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
    if ((long long)n * heads > INT_MAX / 2 || heads / cache->kv_heads > 4096)
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


constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];  // SM count, once the kernels' attributes are set

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
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return SPEC_ERR_CUDA;
        }
        for (const Kernels *k : {&kernels_d64(), &kernels_d128()})
            for (int i = 0; i < 3; ++i)
                for (int f = 0; f < 2; ++f)
                    if (cudaFuncSetAttribute(k->attend[i][f], cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             k->attend_smem[i]) != cudaSuccess ||
                        cudaFuncSetAttribute(k->weigh[i][f], cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             k->weigh_smem[i]) != cudaSuccess) {
                        cudaGetLastError();
                        return SPEC_ERR_CUDA;
                    }
        g_sms[dev].store(v, std::memory_order_release);
    }
    *sms = v;
    return SPEC_OK;
}

// [dim, token, head, page] over the codes; a box is one block of one head.  A
// token's row is one span of the swizzle, as the products read it.
spec_status make_map(const spec_cache &c, void *base, const int64_t stride[3], CUtensorMap *map)
{
    const EncodeTiled encode = encoder();
    if (!encode)
        return SPEC_ERR_CUDA;
    const cuuint64_t size[4] = {(cuuint64_t)c.dim, (cuuint64_t)c.block, (cuuint64_t)c.kv_heads, (cuuint64_t)c.num_pages};
    const cuuint64_t step[3] = {(cuuint64_t)stride[2], (cuuint64_t)stride[1], (cuuint64_t)stride[0]};
    const cuuint32_t box[4] = {(cuuint32_t)c.dim, (cuuint32_t)c.block, 1, 1}, one[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, size, step, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  c.dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? SPEC_OK
               : SPEC_ERR_INVALID_ARG;
}

// Columns of a row tile: the fewest that hold a key head's rows, 48 at most.  (64 columns, with two softmax
// warpgroups, took 5 to 12% longer than 48 with three for trees of 64 nodes and chunks of 1000 tokens; 32 with four
// took 17% longer for the chunks, and 5% less for the trees.)
struct Shape {
    int index, nt, row_tiles;
};
Shape shape_for(const spec_cache &c, int n, int heads)
{
    const int rows = n * (heads / c.kv_heads);
    const int i = rows <= 16 ? 0 : rows <= 32 ? 1 : 2, nt = 16 * (i + 1);
    return {i, nt, (rows + nt - 1) / nt};
}

AttendArgs make_args(const spec_cache *cache, const int32_t *lengths, const void *q, const int64_t q_stride[3], int n,
                     int heads, const spec_cache_form *form, const Shape &shape, uint32_t *status)
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
    a.group = heads / cache->kv_heads;
    a.per_group = a.group == 1 ? 0 : (uint32_t)(((1ull << 32) + a.group - 1) / a.group);
    a.row_tiles = shape.row_tiles;
    a.status = status;
    a.wait_limit = wait_limit();
    return a;
}

bool has_form(const spec_cache_form *f) { return f->softcap > 0.0f || f->slopes; }

// The split queries and their factors; rows of row tiles filled up.
int64_t split_bytes(const spec_cache &c, const Shape &s) { return (int64_t)c.batch * c.kv_heads * s.row_tiles * s.nt * (2 * c.dim + 4); }

// Points the arguments into the workspace and launches split_kernel.
spec_status split_queries(AttendArgs &a, const Shape &s, void *workspace, const Kernels &k, cudaStream_t stream)
{
    const int64_t rows = (int64_t)a.c.batch * a.c.kv_heads * s.row_tiles * s.nt, each = 256 / (a.c.dim / 8) * kSplitRows;
    if (rows > INT_MAX / 2)
        return SPEC_ERR_UNSUPPORTED;
    a.split = (uint8_t *)workspace;
    a.factor = (float *)(a.split + rows * 2 * a.c.dim);
    uint32_t nt = (uint32_t)s.nt;
    void *args[] = {&a, &nt};
    if (cudaLaunchKernel(k.split, dim3((unsigned)((rows + each - 1) / each)), dim3(256), args, 0, stream) != cudaSuccess) {
        cudaGetLastError();
        return SPEC_ERR_CUDA;
    }
    return SPEC_OK;
}

// Launches a kernel that may begin before the one ahead of it in the stream has ended (it waits on the device).
spec_status launch_behind(const void *kernel, dim3 grid, int threads, size_t smem, void **args, cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelExC(&cfg, kernel, args) != cudaSuccess) {
        cudaGetLastError();
        return SPEC_ERR_CUDA;
    }
    return SPEC_OK;
}

int64_t part_bytes(const Shape &s, int dim, int sms) { return 2ll * sms * s.nt * dim * 4; }
int64_t sum_bytes(const Shape &s, int sms) { return 2ll * sms * s.nt * 8; }

}  // namespace

extern "C" {

spec_status spec_cache_set_wait_limit(int clocks)
{
    if (clocks < 0)
        return SPEC_ERR_INVALID_ARG;
    g_wait_limit.store(clocks, std::memory_order_relaxed);
    return SPEC_OK;
}

spec_status spec_cache_attend_workspace(const spec_cache *cache, int n, int heads, int64_t *bytes)
{
    spec_status st = check_cache(cache);
    if (st != SPEC_OK)
        return st;
    if (!bytes || n < 0 || heads < 1 || heads % cache->kv_heads)
        return SPEC_ERR_INVALID_ARG;
    if ((long long)n * heads > INT_MAX / 2)
        return SPEC_ERR_UNSUPPORTED;
    *bytes = 0;
    if (cache->batch == 0 || n == 0)
        return SPEC_OK;
    int sms = 0;
    st = device_sms(&sms);
    if (st != SPEC_OK)
        return st;
    const Shape s = shape_for(*cache, n, heads);
    *bytes = split_bytes(*cache, s) + part_bytes(s, cache->dim, sms) + sum_bytes(s, sms) + 16ll * sms;
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
    if (!out || ((uintptr_t)out & 15u) || bad4(lse, true) || !workspace || ((uintptr_t)workspace & 15u) ||
        workspace_bytes < 0)
        return SPEC_ERR_INVALID_ARG;
    int sms = 0;
    st = device_sms(&sms);
    if (st != SPEC_OK)
        return st;
    const Shape shape = shape_for(*cache, n, heads);
    const int64_t parts = part_bytes(shape, cache->dim, sms), sums = sum_bytes(shape, sms);
    const int64_t split = split_bytes(*cache, shape);
    if (workspace_bytes < split + parts + sums + 16ll * sms)
        return SPEC_ERR_INVALID_ARG;
    AttendArgs a = make_args(cache, lengths, q, q_stride, n, heads, form, shape, status);
    a.out = (__nv_bfloat16 *)out;
    a.lse = lse;
    a.part = (float *)((char *)workspace + split);  // a multiple of 64 bytes in
    a.part_sum = (float2 *)((char *)a.part + parts);
    a.joins = (int4 *)((char *)a.part_sum + sums);
    CUtensorMap kmap, vmap;
    if ((st = make_map(*cache, cache->k, cache->k_stride, &kmap)) != SPEC_OK ||
        (st = make_map(*cache, cache->v, cache->v_stride, &vmap)) != SPEC_OK)
        return st;
    const Kernels &k = cache->dim == 64 ? kernels_d64() : kernels_d128();
    if ((st = split_queries(a, shape, workspace, k, (cudaStream_t)stream)) != SPEC_OK)
        return st;
    void *args[] = {&a, &kmap, &vmap}, *join_args[] = {&a};
    st = launch_behind(k.attend[shape.index][has_form(form)], dim3(sms), k.attend_threads[shape.index],
                       (size_t)k.attend_smem[shape.index], args, (cudaStream_t)stream);
    if (st != SPEC_OK || (long long)cache->max_blocks * cache->block <= kTile)
        return st;  // units of one tile are never in parts
    return launch_behind(k.join[shape.index], dim3(sms, shape.nt / kJoinRows), 32 * kJoinRows, 0, join_args,
                         (cudaStream_t)stream);
}

spec_status spec_cache_weigh(const spec_cache *cache, const int32_t *lengths, const void *q,
                             const int64_t q_stride[3], int n, int heads, const spec_cache_form *form,
                             const float *lse, float *weights, void *workspace, int64_t workspace_bytes,
                             uint32_t *status, void *stream)
{
    NvtxScope nvtx("spec_cache_weigh");
    spec_status st = check_call(cache, lengths, q, q_stride, n, heads, form, status);
    if (st != SPEC_OK || cache->batch == 0 || n == 0)
        return st;
    if (bad4(lse, true) || bad4(weights, true) || !workspace || ((uintptr_t)workspace & 15u))
        return SPEC_ERR_INVALID_ARG;
    int sms = 0;
    st = device_sms(&sms);
    if (st != SPEC_OK)
        return st;
    const Shape shape = shape_for(*cache, n, heads);
    AttendArgs a = make_args(cache, lengths, q, q_stride, n, heads, form, shape, status);
    a.lse_in = lse;
    a.weights = weights;
    if (workspace_bytes < split_bytes(*cache, shape))
        return SPEC_ERR_INVALID_ARG;
    CUtensorMap kmap;
    if ((st = make_map(*cache, cache->k, cache->k_stride, &kmap)) != SPEC_OK)
        return st;
    const Kernels &k = cache->dim == 64 ? kernels_d64() : kernels_d128();
    if ((st = split_queries(a, shape, workspace, k, (cudaStream_t)stream)) != SPEC_OK)
        return st;
    void *args[] = {&a, &kmap};
    return launch_behind(k.weigh[shape.index][has_form(form)], dim3(sms), kWeighThreads, (size_t)k.weigh_smem[shape.index],
                         args, (cudaStream_t)stream);
}

}  // extern "C"
