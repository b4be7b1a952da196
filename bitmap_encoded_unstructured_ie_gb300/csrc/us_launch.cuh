// us_launch.cuh -- launches with programmatic stream serialisation: the kernel may
// start while its predecessor drains, and waits (us::pdl_wait) before it reads.
#pragma once

#include "us_common.cuh"

namespace us {

// args: a pointer to each of the kernel's parameters (us_api.cu)
us_status launch_kernel(const void* kern, dim3 grid, int threads, size_t smem, cudaStream_t st, void** args);

template <class... Params, class... Args>
us_status launch_pdl(void (*kern)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
    auto with = [&](Params... p) {
        void* at[] = {const_cast<void*>(static_cast<const void*>(&p))...};
        return launch_kernel(reinterpret_cast<const void*>(kern), grid, threads, smem, st, at);
    };
    return with(Params(args)...);
}

}  // namespace us
