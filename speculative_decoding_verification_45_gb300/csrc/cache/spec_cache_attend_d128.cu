// Attention and weights over the 8-bit cache for heads of 128.
#include "spec_cache_attend.cuh"

const specc::Kernels &specc::kernels_d128()
{
    static const Kernels k = all_kernels<128>();
    return k;
}
