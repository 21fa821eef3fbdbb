// Attention and weights over the 8-bit cache for heads of 64.
#include "spec_cache_attend.cuh"

const specc::Kernels &specc::kernels_d64()
{
    static const Kernels k = all_kernels<64>();
    return k;
}
