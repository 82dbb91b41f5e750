// Softmax statistics of the vocabulary-split cross entropy, shared by the products that
// leave them (LIN_LSE, LIN_EXP) and the kernel that joins them. Exponents are kept to
// base 2: a logit l counts as l log2(e), and a term is one multiply-add and one ex2.
// Terms are relative to 0 as long as a tile's sum of them is in [2^-64, 2^64] (logits up to
// some 44 either way): float32, and bf16 with the same exponents, hold them as exactly as
// any, no maximum is needed, and terms of different tiles can be used side by side.
#pragma once

#include "activation.cuh"
#include "linear.h"

namespace rtp {

namespace {

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;

__device__ __forceinline__ float minus_infinity() { return __uint_as_float(0xFF800000u); }

// What the terms of a part refer to: its largest logit, or 0 where every one is -inf.
__device__ __forceinline__ float finite_ref(float top) { return top == minus_infinity() ? 0.0f : top; }

struct SoftmaxArgs {
    float2* stats;
    float* target_logit;
    const void* targets;
    const float* weights;
    int64_t vocab, ignore;
    int32_t targets64, parts;  // parts of a row, over all groups
};

// Whether exponentials relative to 0 with this sum are kept (not a NaN sum).
__device__ __forceinline__ bool in_range(float sum) { return sum >= 0x1p-64f && sum <= 0x1p64f; }

// The target of a row, counted over the whole vocabulary.
__device__ __forceinline__ int64_t target_at(const void* targets, int wide, int64_t row)
{
    return wide ? __ldcg(static_cast<const long long*>(targets) + row) : (int64_t)__ldcg(static_cast<const int*>(targets) + row);
}
// The same, counted from column `first`; -1: not in the `cols` columns from there.
__device__ __forceinline__ int target_in(const SoftmaxArgs& a, int64_t row, int64_t first, int cols)
{
    const int64_t t = target_at(a.targets, a.targets64, row) - first;
    return t >= 0 && t < cols ? (int)t : -1;
}
__device__ __forceinline__ bool takes_part(const SoftmaxArgs& a, int64_t row)
{
    return target_at(a.targets, a.targets64, row) != a.ignore && (!a.weights || __ldcg(a.weights + row) != 0.0f);
}
// Columns of the vocabulary from column `first` on, of at most `cols`.
__device__ __forceinline__ int valid_columns(const SoftmaxArgs& a, int64_t first, int cols)
{
    return (int)max((int64_t)0, min((int64_t)cols, a.vocab - first));
}

inline SoftmaxArgs softmax_args(const LinSoftmax& s, int parts)
{
    return SoftmaxArgs{s.stats, s.target_logit, s.targets, s.weights, s.vocab, s.ignore, s.targets64, parts};
}

}  // namespace

}  // namespace rtp
