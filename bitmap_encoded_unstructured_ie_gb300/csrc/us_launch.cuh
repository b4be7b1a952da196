// us_launch.cuh -- launches with programmatic stream serialisation: the kernel may
// start while its predecessor drains, and waits (us::pdl_wait) before it reads.
#pragma once

#include "us_common.cuh"

namespace us {

template <class... Params, class... Args>
us_status launch_pdl(void (*kern)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, Params(args)...) == cudaSuccess ? US_OK : US_ERR_CUDA;
}

}  // namespace us
