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
    LIN_LSE = 3,   // acc = logits: softmax statistics of each row's part of a tile, and the target's logit
    LIN_EXP = 4,   // LIN_LSE, and out = the exponentials that the statistics sum up
};

// Softmax statistics (LIN_LSE, LIN_EXP): for a row and a part (the columns of one tile)
// x = ref, y = sum over the part's columns j of 2^(l_j log2(e) - ref). ref is 0, or,
// where that sum is not in [2^-64, 2^64], the part's largest l_j log2(e); -inf with a sum
// of 0. LIN_EXP writes the terms of the sums, in the rows that take part in gradients
// (target other than `ignore`, weight other than 0), and 0 in the others.
struct LinSoftmax {
    float2* stats = nullptr;        // [rows][groups * parts of a group]
    float* target_logit = nullptr;  // [rows]; not written where the target is in no column
    const void* targets = nullptr;  // [rows], int64 or int32: column counted over the groups
    int targets64 = 1;
    int64_t vocab = 0;              // columns from here on (counted over the groups) take no part
    int64_t ignore = 0;
    const float* weights = nullptr;  // [rows], or NULL: 1
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
    bool accumulate = false;           // gradients in float32: out += product
    const float* row_scale = nullptr;  // b_t gradients: row r of the product times row_scale[r]
    LinEpi epi = LIN_OUT;
    int act = RTP_ACT_NONE;
    int64_t rows = 0, cols = 0, kdim = 0;
    int64_t lda = 0, ldb = 0;  // row strides in elements of A and B as stored, 0: dense
    int64_t ldo = 0;           // LIN_EXP: of out
    int64_t kdims[LIN_MAX_GROUPS] = {};  // b_t, not a_t: K range of a group where it is shorter than kdim (0: kdim)
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
    LinSoftmax softmax;
};

// The 2-SM pair kernel (linear_gemm.cu): any LinGemm, in tiles of 256 x 256 (LIN_GLU:
// 128 columns of the output).
constexpr int LIN_TILE_ROWS = 256, LIN_TILE_COLS = 256;
// Columns of the few-row kernel's tiles.
constexpr int LIN_FEW_COLS = 128;
int launch_linear_gemm(const char* fn, const LinGemm& g, cudaStream_t stream);
// The few-row kernel (linear_few.cu): all but LIN_DGLU, at most
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
