// Internal interface of the products behind rtp_tp_linear and rtp_tp_glu: one
// host description of a launch, and the two kernels that can run it.
#pragma once

#include <cuda_runtime.h>

#include "rtp_internal.h"

namespace rtp {

constexpr int LIN_MAX_GROUPS = 16;  // operand pairs of one launch: 2 per rank (gate and up) of at most 8 ranks
constexpr int LIN_MAX_RANKS = 8;

enum LinEpi : int {
    LIN_OUT = 0,   // out = act(acc + bias) + residual; optionally h = acc + bias
    LIN_GLU = 1,   // out = act(gate) * up, from B (gate) and B2 (up); optionally out2 = gate, out3 = up
    LIN_DGLU = 2,  // acc = dY: out = acc * up * act'(gate), out2 = acc * act(gate); gate = aux, up = aux2
};

// A [rows, kdim] times B [kdim, cols], bf16 row-major, float32 accumulation.
//   groups, fused   `groups` products side by side (group g: A[g] B[g] -> out[g]), or, fused,
//                   their sum in one accumulator (-> out[0])
//   a_t             A is stored [kdim, rows] (its transpose is multiplied)
//   b_t             B is stored [cols, kdim]
//   a_shared        every group multiplies the same A (raster order only)
struct LinGemm {
    int groups = 1;
    bool fused = false, a_t = false, b_t = false, a_shared = false, out_f32 = false;
    LinEpi epi = LIN_OUT;
    int act = RTP_ACT_NONE;
    int64_t rows = 0, cols = 0, kdim = 0;
    const void* A[LIN_MAX_GROUPS] = {};
    const void* B[LIN_MAX_GROUPS] = {};
    const void* B2[LIN_MAX_RANKS] = {};
    void* out[LIN_MAX_GROUPS] = {};
    void* out2[LIN_MAX_RANKS] = {};  // LIN_OUT: h; LIN_GLU: gate; LIN_DGLU: the up gradient
    void* out3[LIN_MAX_RANKS] = {};  // LIN_GLU: up
    const void* bias[LIN_MAX_RANKS] = {};
    const void* residual[LIN_MAX_RANKS] = {};
    const void* aux[LIN_MAX_RANKS] = {};
    const void* aux2[LIN_MAX_RANKS] = {};
};

// The 2-SM pair kernel (linear_gemm.cu): any LinGemm, in tiles of 256 x 256 (LIN_GLU:
// 128 columns of the output).
constexpr int LIN_TILE_ROWS = 256, LIN_TILE_COLS = 256;
int launch_linear_gemm(const char* fn, const LinGemm& g, cudaStream_t stream);
// The few-row kernel (linear_few.cu): LIN_OUT and LIN_GLU, at most
// LIN_FEW_ROWS rows, no transposed operands. weights_ready: nothing queued on the
// stream since a kernel that waited for its own predecessor writes B, so B may be
// read before the previous kernel has finished.
constexpr int LIN_FEW_ROWS = 128;
int launch_linear_few(const char* fn, const LinGemm& g, bool weights_ready, cudaStream_t stream);

// This thread's launches by form (rtp_product_launches).
extern thread_local int32_t product_launches[RTP_PRODUCT_FORMS];

int take_linear_gemm_error(void* stream, uint32_t* code);
int take_linear_split_error(void* stream, uint32_t* code);
int take_linear_few_error(void* stream, uint32_t* code);

}  // namespace rtp
