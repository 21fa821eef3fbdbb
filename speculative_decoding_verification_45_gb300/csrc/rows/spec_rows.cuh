// spec_rows.cuh -- what the kernels of the 8-bit rows share (include/spec_verify.h
// states the operations).
#ifndef SPEC_ROWS_CUH
#define SPEC_ROWS_CUH

#include "../cache/spec_cache.cuh"

namespace specc {

constexpr int kScaleBlock = 128;  // elements of a row with one scale
constexpr int kMaxWidth = SPEC_MAX_ROW;

inline int scale_blocks(int dim) { return (dim + kScaleBlock - 1) / kScaleBlock; }

// Host checks of codes and scales; block_rows: rows with one scale.
inline spec_status check_coded(const spec_coded *c)
{
    if (!c || c->rows < 0 || c->dim < 16 || (c->dim & 15) || c->rows > SPEC_MAX_CODED_ROWS)
        return SPEC_ERR_INVALID_ARG;
    if ((c->code != SPEC_E4M3 && c->code != SPEC_E5M2) || c->dim > kMaxWidth)
        return SPEC_ERR_UNSUPPORTED;
    if (c->rows == 0)
        return SPEC_OK;
    if (!c->codes || ((uintptr_t)c->codes & 15u) || !c->scale || c->stride < c->dim || (c->stride & 15) ||
        c->stride >= (1ll << 40) || c->scale_stride < scale_blocks(c->dim) || c->scale_stride >= (1ll << 40))
        return SPEC_ERR_INVALID_ARG;
    return SPEC_OK;
}

// A matrix of rows in bf16 or fp32: 16-byte aligned, its row stride too.
inline bool bad_rows(const void *p, int64_t stride, int dtype)
{
    const int64_t size = dtype == SPEC_BF16 ? 2 : 4;
    return !p || ((uintptr_t)p & 15u) || ((stride * size) & 15) || stride < 0 || stride >= (1ll << 38);
}
inline bool bad_dtype(int dtype) { return dtype != SPEC_F32 && dtype != SPEC_BF16; }

// Kernels here may begin while the one before them in the stream ends, and let the next one do so: each sets up what it
// can and then waits for everything before it (all threads, ahead of any access to global memory).
__device__ __forceinline__ void after_previous()
{
    asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;" ::: "memory");
}

template <typename... Params, typename... Given>
inline spec_status launch(void (*kernel)(Params...), dim3 grid, int threads, uint32_t smem, int cluster, cudaStream_t stream,
                          const Given &...given)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, Params(given)...) != cudaSuccess) {
        cudaGetLastError();
        return SPEC_ERR_CUDA;
    }
    return SPEC_OK;
}

}  // namespace specc

#endif
