// Launch of a kernel that may be set up while the stream's previous kernel still runs: it
// waits for that one (griddepcontrol.wait) before it touches memory.
#pragma once

#include <cuda_runtime.h>

#include "rtp_internal.h"

namespace rtp {

template <class... A, class... B>
int launch(const char* fn, void (*kernel)(A...), dim3 grid, int threads, cudaStream_t stream, B... args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? RTP_OK : fail(RTP_ECUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
}

}  // namespace rtp
