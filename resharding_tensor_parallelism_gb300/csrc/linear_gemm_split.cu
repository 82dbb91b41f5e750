// The pair products' kernels whose tiles are split along K over a cluster
// (linear_gemm.cuh, SPLIT), in a translation unit of their own.
#include "linear_gemm.cuh"

namespace rtp {

int launch_linear_split(const char* fn, int cfg, LinArgs& a, cudaStream_t stream)
{
    return launch_cfg<true>(fn, cfg, a, stream);
}

int take_linear_split_error(void* stream, uint32_t* code) { return take_tp_error(stream, code); }

}  // namespace rtp
