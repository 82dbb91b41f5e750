// Softmax cross entropy of an output layer whose vocabulary is split over P virtual
// ranks, without the logits: W_i [K, V/P] are the column-parallel shards.
//
//   l = X [W_0 .. W_{P-1}]        lse_r = log sum_j exp l_rj       loss_r = lse_r - l_{r,t_r}
//   d_rj = g_r (exp(l_rj - lse_r) - [j = t_r])     dX = sum_i d_i W_i^T     dW_i = X^T d_i
//
// Forward: the product's epilogue leaves, for each row and tile, the sum of the
// exponentials (softmax.cuh); loss_rows_kernel joins them.
// Training, 6 M K V operations: the same product also writes the exponentials e in bf16,
// all of a row relative to the same number. With s_r the row's sum,
//   d_rj = (g_r / s_r) (e_rj - s_r [j = t_r])
// so the second factor is e but for one element of a row, and the first one is applied to
// the rows of what d multiplies: dX_r = (g_r / s_r) sum_j (..)_rj W_j in that product's
// epilogue, dW = X'^T (..) with X'_r = (g_r / s_r) X_r. loss_rows_kernel writes that element,
// the factor and X'; e is never read but by the two products. (Turning e into d in a pass of
// its own took 0.63 ms of the 16.3 of 8192 x 4096 x 131072, and one more rounding.) Rows with
// logits beyond what exponentials hold relative to 0 are brought to one reference there.
// Recomputing the logits instead of keeping e would cost a third more operations.
//
// The exponentials take 2 V bytes a row. Rows are taken in pieces, so that they take no
// more than the float32 sums of dW that several pieces need (4 K V: 2 K rows), or 1 GiB.
// With several pieces dW is summed in float32, by adds in the output's TMA stores.
//
// The tensor pipe bounds many rows, the weights' bytes few. Measured at 4096 x 131072 on 8
// ranks: 8192 rows forward 5.1 ms (1730 TFLOP/s), training 15.8 to 16.5 (the power cap);
// one row 156 us (6.9 TB/s of the weights).
#include <algorithm>
#include <cstring>

#include "launch.cuh"
#include "linear.h"
#include "softmax.cuh"
#include "tcgen05.cuh"

namespace rtp {

namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;

// Sums of one call, at the start of its workspace.
struct Shared {
    double weight;  // of the counted rows
    float scale;    // of a row's gradient, before its own weight
};
constexpr int64_t SHARED_BYTES = 256;

struct RowsArgs {
    SoftmaxArgs softmax;  // of the piece's rows
    float* loss;          // of the piece's rows
    float* lse;           // or NULL
    // training
    __nv_bfloat16* e[LIN_MAX_RANKS];
    const uint4* x;  // [rows, K], or its copy at `scaled`
    uint4* scaled;   // x times the row's factor
    float* factor;
    Shared* shared;
    int64_t ld;  // of e
    int32_t P, cols, part_cols, parts_of_rank, x_vectors, x_stride, scaled_stride;
};

template <class T, class F>
__device__ __forceinline__ T block_reduce(T v, T* scratch, F&& f)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();  // a previous result has been read
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) v = f(v, scratch[w]);
    return v;
}

__device__ __forceinline__ uint4 times(const uint4& v, float f)
{
    return make_uint4(pack_bf16(bf16_lo(v.x) * f, bf16_hi(v.x) * f), pack_bf16(bf16_lo(v.y) * f, bf16_hi(v.y) * f),
                      pack_bf16(bf16_lo(v.z) * f, bf16_hi(v.z) * f), pack_bf16(bf16_lo(v.w) * f, bf16_hi(v.w) * f));
}

// One row a block: joins the row's statistics into lse and loss and, TRAIN, does what the
// head of this file says. Latency bound (1 to 8 KB of statistics and K elements a row), so
// every load goes out first, and a row whose parts all refer to 0 takes one barrier
// (8192 rows of 512 parts, K = 4096: 60 us with loads where they are used and two
// reductions; a warp a row 54, but 18 instead of 13 for 777 rows of 196).
template <bool TRAIN>
__global__ void __launch_bounds__(THREADS) loss_rows_kernel(const __grid_constant__ RowsArgs a)
{
    __shared__ double scratch[WARPS];
    float* scratch_f = reinterpret_cast<float*>(scratch);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int me = (int)threadIdx.x;
    const int64_t row = blockIdx.x;
    const float2* stats = a.softmax.stats + row * a.softmax.parts;
    const int64_t t = target_at(a.softmax.targets, a.softmax.targets64, row);
    const float logit = __ldcg(a.softmax.target_logit + row);  // nothing where the target is not known
    const float w = !TRAIN ? 0.0f : a.softmax.weights ? __ldcg(a.softmax.weights + row) : 1.0f;
    const float scale = TRAIN ? __ldcg(&a.shared->scale) : 0.0f;
    constexpr int AHEAD = 2;  // vectors of X a thread holds: 4096 elements a block
    uint4 x[AHEAD];
    if constexpr (TRAIN) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (me + k * THREADS < a.x_vectors) x[k] = __ldcg(a.x + row * a.x_stride + me + k * THREADS);
    }
    float sum = 0.0f;
    bool other = false;  // a part that refers to something else
#pragma unroll 4
    for (int i = me; i < a.softmax.parts; i += THREADS) {
        const float2 s = __ldcg(stats + i);
        if (s.x == 0.0f) sum += s.y;
        else if (s.x != minus_infinity()) other = true;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((me & 31) == 0) scratch_f[me >> 5] = sum;
    other = __syncthreads_or(other);
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) sum += scratch_f[k];
    const bool ignored = t == a.softmax.ignore, known = t >= 0 && t < a.softmax.vocab, part = !ignored && w != 0.0f;
    float ref = 0.0f;
    if (other) {  // the row's reference is the largest of its parts'
        float top = minus_infinity();
        for (int i = me; i < a.softmax.parts; i += THREADS) top = fmaxf(top, __ldcg(stats + i).x);
        ref = finite_ref(block_reduce(top, scratch_f, [](float x, float y) { return fmaxf(x, y); }));
        sum = 0.0f;
        for (int i = me; i < a.softmax.parts; i += THREADS) {
            const float2 s = __ldcg(stats + i);
            if (s.x != minus_infinity()) sum += s.y * exp2_fast(s.x - ref);
        }
        sum = block_reduce(sum, scratch_f, [](float x, float y) { return x + y; });
        if (TRAIN && part) {
            for (int i = 0; i < a.P; ++i) {
                uint4* e = reinterpret_cast<uint4*>(a.e[i] + row * a.ld);
                for (int v = me; v < a.cols / 8; v += THREADS) {
                    const float r = __ldcg(stats + i * a.parts_of_rank + 8 * v / a.part_cols).x;
                    if (r != ref) e[v] = times(e[v], exp2_fast(r - ref));
                }
            }
            __syncthreads();
        }
    }
    if (me == 0) {
        const float lse = (ref + log2f(sum)) * LN2;
        if (a.lse) a.lse[row] = lse;
        const float loss = lse - logit;  // rounding may leave it below 0; a NaN stays one
        a.loss[row] = ignored ? 0.0f : !known ? __int_as_float(0x7FC00000) : loss < 0.0f ? 0.0f : loss;
    }
    if constexpr (TRAIN) {
        // A target outside the vocabulary shows. What rounding did to the target's element, the
        // largest of the row, is put right in the factor.
        const float rest = exp2_fast(fmaf(logit, LOG2E, -ref)) - sum;
        const __nv_bfloat16 kept = __float2bfloat16_rn(rest);
        const float turned = __bfloat162float(kept);
        const float factor = !part    ? 0.0f
                             : !known ? __int_as_float(0x7FC00000)
                                      : scale * w / sum * (turned != 0.0f ? rest / turned : 1.0f);
        if (me == 0) {
            a.factor[row] = factor;
            if (part && known) a.e[t / a.cols][row * a.ld + t % a.cols] = kept;
        }
        uint4* scaled = a.scaled + row * a.scaled_stride;
        auto put = [&](int v, const uint4& x) {  // a row without a part is 0 whatever it holds
            scaled[v] = part ? times(x, factor) : make_uint4(0u, 0u, 0u, 0u);
        };
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (me + k * THREADS < a.x_vectors) put(me + k * THREADS, x[k]);
        for (int v = me + AHEAD * THREADS; v < a.x_vectors; v += THREADS) put(v, __ldcg(a.x + row * a.x_stride + v));
    }
}

// Sum over 1024 threads, in the first warp (64-bit adds are slow here: by every thread, 8 us).
__device__ __forceinline__ double block_sum_1024(double s)
{
    __shared__ double sums[32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x >= 32) return 0.0;
    s = sums[threadIdx.x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// The weight of the counted rows, from which the gradients' scale follows, and at the end
// the total. One block each, which run beside the product in front of them: that one has
// waited for all earlier work, and neither touches what the other writes. They end after
// the product all the same, so that the kernel behind need wait for them only. alone: there
// is no such product. (The total by the last block of loss_rows_kernel to finish: a counter
// that 16384 blocks count on took 80 us.)
__global__ void __launch_bounds__(1024) loss_scale_kernel(const void* targets, int targets64, const float* weights, int64_t rows,
                                                          int64_t ignore, int mean, float scale, Shared* sh, float* total, int alone)
{
    if (alone) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    double s = 0.0;
    if (mean)
        for (int64_t r = threadIdx.x; r < rows; r += 1024)
            if (target_at(targets, targets64, r) != ignore) s += weights ? (double)__ldcg(weights + r) : 1.0;
    s = block_sum_1024(s);
    if (threadIdx.x == 0) {
        sh->weight = s;
        sh->scale = !mean ? scale : s != 0.0 ? (float)((double)scale / s) : 0.0f;
        if (rows == 0) *total = 0.0f;
    }
    if (!alone) asm volatile("griddepcontrol.wait;" ::: "memory");
}

__global__ void __launch_bounds__(1024) loss_total_kernel(const float* loss, const void* targets, int targets64,
                                                          const float* weights, int64_t rows, int64_t ignore, int mean,
                                                          const Shared* sh, float* total, int alone)
{
    if (alone) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    double s = 0.0;
    for (int64_t r = threadIdx.x; r < rows; r += 1024) {
        const float w = weights ? __ldcg(weights + r) : 1.0f;  // an ignored row's may be anything
        if (w != 0.0f && target_at(targets, targets64, r) != ignore) s += (double)w * (double)__ldcg(loss + r);
    }
    s = block_sum_1024(s);
    if (threadIdx.x == 0) {
        const double weight = __ldcg(&sh->weight);
        *total = (float)(!mean ? s : weight != 0.0 ? s / weight : 0.0);
    }
    if (!alone) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Rows of X to rows that begin on a 128-byte line: the product reads 128 bytes of a row at
// a time, and where those lie across two lines its operands come at two thirds of the rate.
__global__ void __launch_bounds__(THREADS) align_rows_kernel(const uint4* x, uint4* to, int64_t rows, int vectors, int stride)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t n = rows * vectors;
#pragma unroll 2
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < n; i += (int64_t)gridDim.x * THREADS)
        to[i / vectors * stride + i % vectors] = __ldcg(x + i);
}

// dX from the float32 products of its slices (dx_slices), in their order, times the rows' factors.
struct SliceArgs {
    const float4* from;  // [slices][rows][quads]
    const float* factor;
    void* to;
    int64_t quads;  // of all rows
    int32_t row_quads, slices;
};
template <bool F32>
__global__ void __launch_bounds__(THREADS) slices_kernel(const __grid_constant__ SliceArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < a.quads; i += (int64_t)gridDim.x * THREADS) {
        float4 s = __ldcg(a.from + i);
#pragma unroll 8
        for (int k = 1; k < a.slices; ++k) {
            const float4 v = __ldcg(a.from + k * a.quads + i);
            s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        const float f = __ldcg(a.factor + i / a.row_quads);
        s = make_float4(s.x * f, s.y * f, s.z * f, s.w * f);
        if constexpr (F32) static_cast<float4*>(a.to)[i] = s;
        else static_cast<uint2*>(a.to)[i] = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    }
}

// float32 sums to bf16 gradients.
struct RoundArgs {
    const float4* from[LIN_MAX_RANKS];
    uint2* to[LIN_MAX_RANKS];
    int64_t quads;
};
__global__ void __launch_bounds__(THREADS) round_kernel(const __grid_constant__ RoundArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const float4* from = a.from[blockIdx.y];
    uint2* to = a.to[blockIdx.y];
    const int64_t stride = (int64_t)gridDim.x * THREADS;
#pragma unroll 4
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < a.quads; i += stride) {
        const float4 v = __ldcs(from + i);
        to[i] = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    }
}

// ---- host side --------------------------------------------------------------------

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

struct Shape {
    int P;
    int64_t M, K, V, vocab, Vp;
    int64_t lde, ldx;  // row strides of the exponentials and the scaled X: whole lines, which a product reads 128 bytes of
    int64_t piece;  // rows of a piece
    int pieces;
};

// part_cols of the product that a piece of `rows` rows takes
int part_cols(int64_t rows) { return rows <= LIN_FEW_ROWS ? LIN_FEW_COLS : LIN_TILE_COLS; }
int64_t parts(const Shape& s, int64_t rows) { return s.P * ((s.Vp + part_cols(rows) - 1) / part_cols(rows)); }

// Columns of rank i that are in the vocabulary. The products for dX go no further: the exponentials behind are 0, but
// the weights there may be anything, and 0 times an infinity or a NaN is a NaN.
int64_t rank_columns(const Shape& s, int i) { return std::max<int64_t>(0, std::min(s.Vp, s.vocab - i * s.Vp)); }

// Slices of each rank's columns whose products for dX are summed by a kernel of their own
// (0: none, all ranks in one accumulator). dX of few rows and a narrow model has few tiles,
// each the product of the whole vocabulary, which a cluster shares four ways at most:
// 256 x 512 from 8192 columns took 20 us on 8 of 76 pairs. K blocks take 0.28 us of a
// pair, the sum 5 us. Workspaces are sized without a device, so the rule is one for these
// SLICE_PAIRS; a device with fewer SMs, where its slices would not run side by side, takes none.
constexpr int SLICE_PAIRS = 76;
int64_t slice_columns(const Shape& s, int n) { return up((s.Vp + n - 1) / n, 64); }
int dx_slices(const Shape& s, int64_t rows)
{
    if (rows <= 0) return 0;
    const int64_t tiles = ((rows + LIN_TILE_ROWS - 1) / LIN_TILE_ROWS) * ((s.K + LIN_TILE_COLS - 1) / LIN_TILE_COLS);
    const int64_t kbs = s.P * ((s.Vp + 63) / 64);
    const double one = 0.28 * (double)kbs / (double)std::min<int64_t>(4, std::max<int64_t>(1, SLICE_PAIRS / tiles));
    int best = 1;
    double least = one;
    for (int n = 1; n <= LIN_MAX_GROUPS / s.P; ++n) {
        const int64_t parts = tiles * s.P * n, split = std::min<int64_t>(4, SLICE_PAIRS / parts), kdim = slice_columns(s, n);
        if (s.P * n < 2 || split < 1 || kdim < 512 || (n - 1) * kdim >= s.Vp) continue;
        const double t = 0.28 * (double)(kdim / 64) / (double)split + 5.0;
        if (t < 0.9 * least) least = t, best = n;
    }
    return least < one ? best : 0;
}

// Whether the product reads a copy of X with aligned rows: where its gain, an eighth of the
// product's time, is more than the copy's 3 us.
bool aligns_x(const Shape& s, int64_t rows)
{
    return s.K % 64 && rows > LIN_FEW_ROWS && (double)rows * (double)s.K * (double)s.V >= 2e10;
}

int check_shape(const char* fn, int P, int64_t M, int64_t K, int64_t V, int64_t vocab, int64_t piece_rows, bool train, Shape* s)
{
    if (P < 1 || P > LIN_MAX_RANKS) return fail(RTP_EUNSUPPORTED, "%s: P = %d outside [1, %d]", fn, P, LIN_MAX_RANKS);
    const int64_t lim = (int64_t)1 << 31;
    if (M < 0 || M >= lim || K < 1 || K >= lim || V < 1 || V >= lim)
        return fail(RTP_ESHAPE, "%s: sizes M=%lld, K=%lld, V=%lld outside [0 or 1, 2^31)", fn, (long long)M, (long long)K, (long long)V);
    if (V % P || K % 8 || (V / P) % 8)
        return fail(RTP_ESHAPE, "%s: K=%lld and a rank's columns (V=%lld over P=%d) must be multiples of 8 (16-byte rows)", fn,
                    (long long)K, (long long)V, P);
    const double limit = 0x1p50;  // of rows or K times columns: no byte count below overflows
    if ((double)M * (double)V > limit || (double)K * (double)V > limit)
        return fail(RTP_ESHAPE, "%s: M=%lld, K=%lld, V=%lld are too large", fn, (long long)M, (long long)K, (long long)V);
    if (vocab < 1 || vocab > V) return fail(RTP_ESHAPE, "%s: vocab=%lld outside [1, V=%lld]", fn, (long long)vocab, (long long)V);
    if (piece_rows < 0) return fail(RTP_EINVAL, "%s: piece_rows=%lld", fn, (long long)piece_rows);
    s->P = P, s->M = M, s->K = K, s->V = V, s->vocab = vocab, s->Vp = V / P;
    s->lde = up(s->Vp, 64), s->ldx = up(K, 64);
    // As many rows as the head of this file allows, in pieces of about the same size;
    // whole row tiles, so that only the last piece ends inside one.
    const int64_t wanted = piece_rows ? piece_rows : std::max({2 * K, (int64_t)2048, ((int64_t)1 << 29) / V});
    const int64_t most = up(std::min(wanted, std::max<int64_t>(M, 1)), LIN_TILE_ROWS);
    s->pieces = train && M > most ? (int)((M + most - 1) / most) : 1;
    s->piece = s->pieces > 1 ? up((M + s->pieces - 1) / s->pieces, LIN_TILE_ROWS) : M;
    if (s->pieces > 1) s->pieces = (int)((M + s->piece - 1) / s->piece);
    return RTP_OK;
}

// Where things are in a workspace; sum: float32 sums of dW.
struct Space {
    int64_t logit, factor, stats, x, e, slices, sum, bytes;
};
Space space_of(const Shape& s, bool train, bool sum)
{
    // the last piece may be of few rows, with narrower parts than the others
    const int64_t last = s.M - (s.pieces - 1) * s.piece;
    const int64_t most = std::max(s.piece * parts(s, s.piece), last * parts(s, last));
    Space w;
    w.logit = SHARED_BYTES;
    w.factor = w.logit + up(s.piece * 4, 256);
    w.stats = w.factor + (train ? up(s.piece * 4, 256) : 0);
    w.x = w.stats + up(most * 8, 256);
    w.e = w.x + (train || aligns_x(s, s.piece) ? up(s.piece * s.ldx * 2, 256) : 0);
    w.slices = w.e + (train ? up(s.P * s.piece * s.lde * 2, 256) : 0);
    int64_t sliced = 0;
    for (int64_t rows : {s.piece, last}) sliced = std::max(sliced, dx_slices(s, rows) * s.P * rows * s.K * 4);
    w.sum = w.slices + (train ? up(sliced, 256) : 0);
    w.bytes = w.sum + (sum ? s.K * s.V * 4 : 0);
    return w;
}

int check_ptr(const char* fn, const char* name, const void* p, uintptr_t align, bool needed)
{
    if (needed && !p) return fail(RTP_EINVAL, "%s: NULL %s", fn, name);
    if ((uintptr_t)p & (align - 1)) return fail(RTP_EINVAL, "%s: %s must be %d-byte aligned", fn, name, (int)align);
    return RTP_OK;
}
int check_ptrs(const char* fn, const char* name, const void* const* p, int n)
{
    if (!p) return fail(RTP_EINVAL, "%s: NULL %s", fn, name);
    for (int i = 0; i < n; ++i) TRY(check_ptr(fn, name, p[i], 16, true));
    return RTP_OK;
}

struct Call {
    const char* fn;
    Shape s;
    const void* X;
    const void* const* W;
    const void* targets;
    int targets64;
    int64_t ignore;
    char* ws;
    Space space;
};

int check_call(Call& c, int targets64, int64_t workspace_bytes, const float* loss)
{
    const char* fn = c.fn;
    const bool some = c.s.M > 0;
    if (targets64 != 0 && targets64 != 1) return fail(RTP_EINVAL, "%s: targets64 = %d", fn, targets64);
    TRY(check_ptrs(fn, "weight", c.W, c.s.P));
    TRY(check_ptr(fn, "X", c.X, 16, some));
    TRY(check_ptr(fn, "targets", c.targets, targets64 ? 8 : 4, some));
    TRY(check_ptr(fn, "loss", loss, 4, some));
    TRY(check_ptr(fn, "workspace", c.ws, 256, true));
    if (workspace_bytes < c.space.bytes)
        return fail(RTP_EINVAL, "%s: a workspace of %lld bytes, %lld needed", fn, (long long)workspace_bytes, (long long)c.space.bytes);
    return RTP_OK;
}

const void* rows_of(const void* p, int64_t first, int64_t row_bytes)
{
    return p ? static_cast<const char*>(p) + first * row_bytes : nullptr;
}

// The product with its statistics for `rows` rows from `first`, and the rows' arguments.
int softmax_product(const Call& c, LinEpi epi, const float* weights, int64_t first, int64_t rows, RowsArgs* a, cudaStream_t stream)
{
    const void* x = rows_of(c.X, first, c.s.K * 2);
    int64_t ldx = c.s.K;
    if (aligns_x(c.s, rows)) {
        void* to = c.ws + c.space.x;
        ldx = c.s.ldx;
        int sms = 0;
        if (device_sms(&sms)) return fail(RTP_ECUDA, "%s: no CUDA device", c.fn);
        const int64_t vectors = rows * (c.s.K / 8);
        const unsigned blocks = (unsigned)std::min<int64_t>((vectors + THREADS - 1) / THREADS, (int64_t)8 * sms);
        TRY(launch(c.fn, align_rows_kernel, dim3(blocks), THREADS, stream, static_cast<const uint4*>(x), static_cast<uint4*>(to), rows,
                   (int)(c.s.K / 8), (int)(ldx / 8)));
        x = to;
    }
    a->x = static_cast<const uint4*>(x);
    a->x_vectors = (int)(c.s.K / 8);
    a->x_stride = (int)(ldx / 8);
    LinGemm g;
    g.epi = epi;
    g.lda = ldx;
    g.groups = c.s.P;
    g.a_shared = true;
    g.rows = rows;
    g.cols = c.s.Vp;
    g.kdim = c.s.K;
    for (int i = 0; i < c.s.P; ++i) {
        g.A[i] = x;
        g.B[i] = c.W[i];
        if (epi == LIN_EXP) {
            g.out[i] = c.ws + c.space.e + i * rows * c.s.lde * 2;
            g.ldo = c.s.lde;
            a->e[i] = static_cast<__nv_bfloat16*>(g.out[i]);
        }
    }
    g.softmax.stats = reinterpret_cast<float2*>(c.ws + c.space.stats);
    g.softmax.target_logit = reinterpret_cast<float*>(c.ws + c.space.logit);
    g.softmax.targets = rows_of(c.targets, first, c.targets64 ? 8 : 4);
    g.softmax.targets64 = c.targets64;
    g.softmax.vocab = c.s.vocab;
    g.softmax.ignore = c.ignore;
    g.softmax.weights = weights ? weights + first : nullptr;
    a->softmax = softmax_args(g.softmax, (int)parts(c.s, rows));
    a->P = c.s.P;
    a->ld = c.s.lde;
    a->cols = (int)c.s.Vp;
    a->part_cols = part_cols(rows);
    a->parts_of_rank = a->softmax.parts / c.s.P;
    return rows <= LIN_FEW_ROWS ? launch_linear_few(c.fn, g, false, stream) : launch_linear_gemm(c.fn, g, stream);
}

int forward_impl(Call& c, int targets64, int64_t workspace_bytes, float* loss, float* lse, cudaStream_t stream)
{
    c.space = space_of(c.s, false, false);
    TRY(check_call(c, targets64, workspace_bytes, loss));
    TRY(check_ptr(c.fn, "lse", lse, 4, false));
    if (c.s.M == 0) return RTP_OK;
    RowsArgs a = {};
    TRY(softmax_product(c, LIN_LSE, nullptr, 0, c.s.M, &a, stream));
    a.loss = loss;
    a.lse = lse;
    return launch(c.fn, loss_rows_kernel<false>, dim3((unsigned)c.s.M), THREADS, stream, a);
}

int train_impl(Call& c, int targets64, int64_t workspace_bytes, const float* weights, int mean, float scale, float* total,
               float* loss, int dx_dtype, void* dX, int dw_dtype, void* const* dW, int accumulate, cudaStream_t stream)
{
    const char* fn = c.fn;
    const Shape& s = c.s;
    const bool some = s.M > 0;
    if ((dx_dtype != RTP_F32 && dx_dtype != RTP_BF16) || (dw_dtype != RTP_F32 && dw_dtype != RTP_BF16))
        return fail(RTP_EINVAL, "%s: a gradient is of unknown type", fn);
    if (mean != 0 && mean != 1) return fail(RTP_EINVAL, "%s: mean = %d", fn, mean);
    if (accumulate != 0 && accumulate != 1) return fail(RTP_EINVAL, "%s: accumulate = %d", fn, accumulate);
    if (accumulate && (!dW || dw_dtype != RTP_F32)) return fail(RTP_EINVAL, "%s: only float32 weight gradients accumulate", fn);
    const bool sums = dW && dw_dtype == RTP_BF16 && s.pieces > 1;
    c.space = space_of(s, true, sums);
    TRY(check_call(c, targets64, workspace_bytes, loss));
    TRY(check_ptr(fn, "weights", weights, 4, false));
    TRY(check_ptr(fn, "total", total, 4, true));
    TRY(check_ptr(fn, "dX", dX, 16, false));
    if (dW) TRY(check_ptrs(fn, "dW", const_cast<const void* const*>(dW), s.P));
    int sms = 0;
    if (device_sms(&sms)) return fail(RTP_ECUDA, "%s: no CUDA device", fn);
    const int64_t dx_size = dx_dtype == RTP_F32 ? 4 : 2, dw_size = dw_dtype == RTP_F32 ? 4 : 2;
    Shared* sh = reinterpret_cast<Shared*>(c.ws);
    auto set_scale = [&] {
        return launch(fn, loss_scale_kernel, dim3(1), 1024, stream, c.targets, c.targets64, weights, s.M, c.ignore, mean, scale, sh,
                      total, some ? 0 : 1);
    };
    if (!some) {
        TRY(set_scale());
        for (int i = 0; dW && !accumulate && i < s.P; ++i)
            if (cudaMemsetAsync(dW[i], 0, (size_t)(s.K * s.Vp * dw_size), stream) != cudaSuccess)
                return fail(RTP_ECUDA, "%s: cudaMemsetAsync failed", fn);
        return RTP_OK;
    }
    auto sum_up = [&](int piece, int alone) {  // behind the last piece's losses
        if (piece < s.pieces - 1) return (int)RTP_OK;
        return launch(fn, loss_total_kernel, dim3(1), 1024, stream, (const float*)loss, c.targets, c.targets64, weights, s.M, c.ignore,
                      mean, (const Shared*)sh, total, alone);
    };
    for (int p = 0; p < s.pieces; ++p) {
        const int64_t first = p * s.piece, rows = std::min(s.piece, s.M - first);
        RowsArgs a = {};
        TRY(softmax_product(c, LIN_EXP, weights, first, rows, &a, stream));
        if (p == 0) TRY(set_scale());
        a.scaled = reinterpret_cast<uint4*>(c.ws + c.space.x);
        a.scaled_stride = (int)(s.ldx / 8);
        a.factor = reinterpret_cast<float*>(c.ws + c.space.factor);
        a.loss = loss + first;
        a.shared = sh;
        TRY(launch(fn, loss_rows_kernel<true>, dim3((unsigned)rows), THREADS, stream, a));
        const int slices = sms >= 2 * SLICE_PAIRS ? dx_slices(s, rows) : 0;
        if (dX && slices) {
            LinGemm g;
            g.groups = 0;
            g.b_t = true;
            g.out_f32 = true;
            g.rows = rows;
            g.cols = s.K;
            g.kdim = slice_columns(s, slices);
            g.lda = s.lde;
            g.ldb = s.Vp;
            float* products = reinterpret_cast<float*>(c.ws + c.space.slices);
            for (int i = 0; i < s.P; ++i)
                for (int64_t col = 0; col < rank_columns(s, i); col += g.kdim) {
                    const int at = g.groups++;
                    g.A[at] = a.e[i] + col;
                    g.B[at] = static_cast<const __nv_bfloat16*>(c.W[i]) + col;
                    g.kdims[at] = std::min(g.kdim, rank_columns(s, i) - col);
                    g.out[at] = products + at * rows * s.K;
                }
            TRY(launch_linear_gemm(fn, g, stream));
            TRY(sum_up(p, 0));
            const SliceArgs b = {reinterpret_cast<const float4*>(products), a.factor, static_cast<char*>(dX) + first * s.K * dx_size,
                                 rows * s.K / 4, (int)(s.K / 4), g.groups};
            const unsigned blocks = (unsigned)std::min<int64_t>((b.quads + THREADS - 1) / THREADS, (int64_t)8 * sms);
            TRY(launch(fn, dx_dtype == RTP_F32 ? slices_kernel<true> : slices_kernel<false>, dim3(blocks), THREADS, stream, b));
        } else if (dX) {
            LinGemm g;
            g.groups = 0;
            g.fused = true;
            g.b_t = true;
            g.out_f32 = dx_dtype == RTP_F32;
            g.rows = rows;
            g.cols = s.K;
            g.kdim = s.Vp;
            for (int i = 0; i < s.P; ++i) {
                if (!rank_columns(s, i)) continue;
                g.A[g.groups] = a.e[i];
                g.B[g.groups] = c.W[i];
                g.kdims[g.groups++] = rank_columns(s, i);
            }
            g.lda = s.lde;
            g.ldb = s.Vp;
            g.row_scale = a.factor;
            g.out[0] = static_cast<char*>(dX) + first * s.K * dx_size;
            TRY(launch_linear_gemm(fn, g, stream));
            TRY(sum_up(p, 0));
        }
        if (dW) {
            LinGemm g;
            g.groups = s.P;
            g.a_t = true;
            g.a_shared = true;
            g.out_f32 = sums || dw_dtype == RTP_F32;
            g.accumulate = accumulate || p > 0;
            g.lda = s.ldx;
            g.ldb = s.lde;
            g.rows = s.K;
            g.cols = s.Vp;
            g.kdim = rows;
            for (int i = 0; i < s.P; ++i) {
                g.A[i] = a.scaled;
                g.B[i] = a.e[i];
                g.out[i] = sums ? c.ws + c.space.sum + i * s.K * s.Vp * 4 : dW[i];
            }
            TRY(launch_linear_gemm(fn, g, stream));
        }
        if (!dX) TRY(sum_up(p, 1));
    }
    if (sums) {
        RoundArgs a = {};
        for (int i = 0; i < s.P; ++i) {
            a.from[i] = reinterpret_cast<const float4*>(c.ws + c.space.sum + i * s.K * s.Vp * 4);
            a.to[i] = static_cast<uint2*>(dW[i]);
        }
        a.quads = s.K * s.Vp / 4;
        const int64_t blocks = std::min<int64_t>((a.quads + THREADS - 1) / THREADS, (int64_t)8 * sms);
        TRY(launch(fn, round_kernel, dim3((unsigned)blocks, (unsigned)s.P), THREADS, stream, a));
    }
    return RTP_OK;
}

}  // namespace

}  // namespace rtp

using namespace rtp;

extern "C" {

int rtp_tp_cross_entropy_workspace(int P, int64_t M, int64_t K, int64_t V, int64_t piece_rows, int train, rtp_dtype dw_dtype,
                                   int64_t* bytes)
{
    const char* fn = "rtp_tp_cross_entropy_workspace";
    if (!bytes) return fail(RTP_EINVAL, "%s: NULL argument", fn);
    Shape s;
    TRY(check_shape(fn, P, M, K, V, V, piece_rows, train != 0, &s));
    *bytes = space_of(s, train != 0, train && dw_dtype == RTP_BF16 && s.pieces > 1).bytes;
    return RTP_OK;
}

int rtp_tp_cross_entropy(int P, int64_t M, int64_t K, int64_t V, int64_t vocab, const void* X, const void* const* W_shards,
                         int targets64, const void* targets, int64_t ignore_index, void* workspace, int64_t workspace_bytes,
                         float* loss, float* lse, rtp_stream stream)
{
    const char* fn = "rtp_tp_cross_entropy";
    return guarded(fn, [&] {
        Call c = {fn, {}, X, W_shards, targets, targets64, ignore_index, static_cast<char*>(workspace), {}};
        TRY(check_shape(fn, P, M, K, V, vocab, 0, false, &c.s));
        return forward_impl(c, targets64, workspace_bytes, loss, lse, static_cast<cudaStream_t>(stream));
    });
}

int rtp_tp_cross_entropy_train(int P, int64_t M, int64_t K, int64_t V, int64_t vocab, const void* X,
                               const void* const* W_shards, int targets64, const void* targets, int64_t ignore_index,
                               const float* weights, int mean, float scale, int64_t piece_rows, void* workspace,
                               int64_t workspace_bytes, float* total, float* loss, rtp_dtype dx_dtype, void* dX,
                               rtp_dtype dw_dtype, void* const* dW, int accumulate, rtp_stream stream)
{
    const char* fn = "rtp_tp_cross_entropy_train";
    return guarded(fn, [&] {
        Call c = {fn, {}, X, W_shards, targets, targets64, ignore_index, static_cast<char*>(workspace), {}};
        TRY(check_shape(fn, P, M, K, V, vocab, piece_rows, true, &c.s));
        return train_impl(c, targets64, workspace_bytes, weights, mean, scale, total, loss, dx_dtype, dX, dw_dtype, dW, accumulate,
                          static_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
