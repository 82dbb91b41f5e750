// Entry points of the tensor-parallel linear layer and the gated feed-forward
// block: argument checks, choice of kernel, launch order, and the backward's
// element-wise step with the bias gradient.
#include <cstring>
#include <type_traits>

#include "activation.cuh"
#include "linear.h"
#include "tcgen05.cuh"

namespace rtp {

namespace {

// dH = dOut * act'(H) in bf16, and db = column sums of the unrounded dH.
// Reads dOut and H and writes dH once; GELU's arithmetic keeps it below the HBM rate
// (4096 x 16384: 84.7 us, 403 MB at 4750 GB/s; with erff and expf 168). A cluster of 8 blocks takes a strip
// of COLS columns, the blocks taking the rows in turn; a thread owns 8 columns
// (16-byte loads), sums them in float32 over its rows, and the block's row lanes,
// then the cluster's 8 blocks over distributed shared memory, are added in a fixed
// order. Strips of 256 columns (512 bytes of a row) where there are enough of them
// for the GPU, of 64 otherwise.
constexpr int SUM_THREADS = 256, SUM_SPLIT = 8;

struct SumArgs {
    const __nv_bfloat16* dout[LIN_MAX_RANKS];
    const __nv_bfloat16* h[LIN_MAX_RANKS];
    __nv_bfloat16* dh[LIN_MAX_RANKS];
    float* db[LIN_MAX_RANKS];
    int64_t rows;
    int32_t cols, act;
};

template <int COLS>
__global__ void __launch_bounds__(SUM_THREADS) act_grad_kernel(const __grid_constant__ SumArgs a)
{
    constexpr int COL_LANES = COLS / 8, ROW_LANES = SUM_THREADS / COL_LANES;
    __shared__ float part[ROW_LANES][COLS + 1];
    __shared__ float sums[COLS];
    const int g = blockIdx.z, cr = (int)cluster_rank();
    const int cl = threadIdx.x % COL_LANES, rl = threadIdx.x / COL_LANES;
    const int col = (int)blockIdx.x * COLS + cl * 8;
    const bool in = col < a.cols;
    const bool has_h = a.h[g] != nullptr;
    float sum[8] = {};
    if (in) {
        with_act(has_h ? a.act : RTP_ACT_NONE, [&](auto tag) {
            constexpr int ACT = decltype(tag)::value;
#pragma unroll 4
            for (int64_t r = cr * ROW_LANES + rl; r < a.rows; r += ROW_LANES * SUM_SPLIT) {
                const int64_t at = r * a.cols + col;
                const uint4 d = __ldg(reinterpret_cast<const uint4*>(a.dout[g] + at));
                float v[8] = {bf16_lo(d.x), bf16_hi(d.x), bf16_lo(d.y), bf16_hi(d.y),
                              bf16_lo(d.z), bf16_hi(d.z), bf16_lo(d.w), bf16_hi(d.w)};
                if constexpr (ACT != RTP_ACT_NONE) {
                    const uint4 h = __ldg(reinterpret_cast<const uint4*>(a.h[g] + at));
                    const float x[8] = {bf16_lo(h.x), bf16_hi(h.x), bf16_lo(h.y), bf16_hi(h.y),
                                        bf16_lo(h.z), bf16_hi(h.z), bf16_lo(h.w), bf16_hi(h.w)};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float av, dv;
                        act_both<ACT>(x[j], av, dv);
                        v[j] *= dv;
                    }
                    *reinterpret_cast<uint4*>(a.dh[g] + at) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                                         pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += v[j];
            }
        });
    }
    if (!a.db[g]) return;  // uniform over the cluster
#pragma unroll
    for (int j = 0; j < 8; ++j) part[rl][cl * 8 + j] = sum[j];
    __syncthreads();
    if (threadIdx.x < COLS) {
        float s = 0.0f;
        for (int r = 0; r < ROW_LANES; ++r) s += part[r][threadIdx.x];
        sums[threadIdx.x] = s;
    }
    cluster_sync();
    const int c = (int)blockIdx.x * COLS + (int)threadIdx.x;
    if (cr == 0 && threadIdx.x < COLS && c < a.cols) {
        float s = 0.0f;
        for (int r = 0; r < SUM_SPLIT; ++r) {
            float v;
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(v)
                         : "r"(map_to_rank(smem_u32(&sums[threadIdx.x]), (uint32_t)r))
                         : "memory");
            s += v;
        }
        a.db[g][c] = s;
    }
    cluster_sync();  // no block leaves while block 0 reads its sums
}

int launch_act_grad(const char* fn, const SumArgs& a, int groups, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = SUM_SPLIT;
    attr[0].val.clusterDim.z = 1;
    const bool wide = (int64_t)(a.cols / 256) * SUM_SPLIT * groups >= 256;
    const int cols = wide ? 256 : 64;
    cfg.gridDim = dim3((unsigned)((a.cols + cols - 1) / cols), SUM_SPLIT, (unsigned)groups);
    cfg.blockDim = dim3(SUM_THREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = wide ? cudaLaunchKernelEx(&cfg, act_grad_kernel<256>, a) : cudaLaunchKernelEx(&cfg, act_grad_kernel<64>, a);
    if (e != cudaSuccess) return fail(RTP_ECUDA, "%s: activation gradient launch failed: %s", fn, cudaGetErrorString(e));
    return RTP_OK;
}

// The same product's rows from `first` on.
LinGemm rows_from(const LinGemm& p, int64_t first)
{
    LinGemm r = p;
    r.rows = p.rows - first;
    auto shift = [first](auto& q, int64_t row_bytes) {
        if (q) q = (std::remove_reference_t<decltype(q)>)((uintptr_t)q + (uintptr_t)(first * row_bytes));
    };
    for (int g = 0; g < LIN_MAX_GROUPS; ++g) {
        shift(r.A[g], p.kdim * 2);
        shift(r.out[g], p.cols * (p.out_f32 ? 4 : 2));
    }
    for (int g = 0; g < LIN_MAX_RANKS; ++g) {
        shift(r.out2[g], p.cols * 2);
        shift(r.out3[g], p.cols * 2);
        shift(r.residual[g], p.cols * 2);
    }
    return r;
}

// Rows behind the last whole row tile that the few-row kernel takes (0: none). The pair
// kernel multiplies a nearly empty row tile like a full one; where these tiles begin a
// wave of their own, the weights read once more cost less than that wave. Pair kernel
// alone -> both, 1 and 48 rows over: 768 x 4096 x 6144 (24 column tiles) 47.5 -> 39.3 and
// 41.3 us, 1024 x 16384 x 4096 (16) 158 -> 108 and 111, 2304 x 2048 x 2048 (8) 28.8 -> 25.8
// and 27.0. The other side: 2048 x 4096 x 9728 (38) 109 -> 113 and 117, 1024 x 1024 x 4096
// (16, 16 K blocks) 20.5 -> 19.9 and 21.0; with 96 and 128 rows over most of the gain is gone.
// At the limits (64 rows, 25 column tiles, 32 K blocks) 28.8 -> 29.4. Between 25 and 38
// column tiles (4 to 8 row tiles, 1 and 64 rows over) 32 K blocks come out even or lose:
// 30 tiles 38.9 -> 39.5 and 39.0 -> 40.9 us, 36 tiles 38.7 -> 39.1 and 39.0 -> 41.2; with 64 K
// blocks both would still gain, 64.9 -> 57.7 and 65.3 -> 60.2, 84.6 -> 80.2 and 84.8 -> 82.4.
// The limit on column tiles is the one that holds for every K.
int64_t rest_rows(const LinGemm& p)
{
    constexpr int64_t MAX_REST = 64, MIN_K = 32 * 64;
    const int64_t rest = p.rows % LIN_TILE_ROWS, m_tiles = p.rows / LIN_TILE_ROWS;
    const int64_t k = p.kdim * (p.fused ? p.groups : 1);
    int sms = 0;
    if (!rest || rest > MAX_REST || !m_tiles || k < MIN_K || device_sms(&sms) || sms < 2) return 0;
    const int64_t pairs = sms / 2, tile_cols = p.epi == LIN_GLU ? LIN_TILE_COLS / 2 : LIN_TILE_COLS;
    const int64_t n_tiles = (p.fused ? 1 : p.groups) * ((p.cols + tile_cols - 1) / tile_cols);
    if (3 * n_tiles > pairs) return 0;
    const int64_t waves = (n_tiles * (m_tiles + 1) + pairs - 1) / pairs;
    return waves > (n_tiles * m_tiles + pairs - 1) / pairs ? rest : 0;
}

// A forward product: the few-row kernel up to LIN_FEW_ROWS rows, the pair kernel
// beyond, or both (rest_rows). Few-row time over pair time, products of 2048 x 2048 to 8192 x 28672: 0.57 to
// 0.88 at 48 rows, 0.73 to 0.99 at 96, 0.78 to 1.04 at 128 (the largest: 88 us against
// 93; 4096 x 16384 on 8 ranks: 32.4 against 31.4).
int forward(const char* fn, const LinGemm& p, bool weights_ready, cudaStream_t stream)
{
    if (p.rows <= LIN_FEW_ROWS) return launch_linear_few(fn, p, weights_ready, stream);
    const int64_t rest = rest_rows(p);
    if (!rest) return launch_linear_gemm(fn, p, stream);
    LinGemm top = p;
    top.rows = p.rows - rest;
    int st = launch_linear_gemm(fn, top, stream);
    // the pair kernel waits for its predecessors and does not write B, so B is ready
    return st ? st : launch_linear_few(fn, rows_from(p, top.rows), true, stream);
}

#define TRY(call)          \
    do {                   \
        int st_ = (call);  \
        if (st_) return st_; \
    } while (0)

int check_common(const char* fn, int P, int64_t M, int64_t a, int64_t b, int act)
{
    if (P < 1 || P > LIN_MAX_RANKS) return fail(RTP_EUNSUPPORTED, "%s: P = %d outside [1, %d]", fn, P, LIN_MAX_RANKS);
    if (act < RTP_ACT_NONE || act > RTP_ACT_RELU) return fail(RTP_EINVAL, "%s: unknown activation %d", fn, act);
    const int64_t lim = (int64_t)1 << 31;
    if (M < 0 || a < 1 || b < 1 || M >= lim || a >= lim || b >= lim)
        return fail(RTP_ESHAPE, "%s: sizes M=%lld, %lld, %lld outside [0 or 1, 2^31)", fn, (long long)M, (long long)a, (long long)b);
    return RTP_OK;
}

int check_dtype(const char* fn, const char* what, int dtype)
{
    if (dtype != RTP_F32 && dtype != RTP_BF16) return fail(RTP_EINVAL, "%s: %s is of unknown type %d", fn, what, dtype);
    return RTP_OK;
}

// Every pointer of an array of n is there and 16-byte aligned (not needed: may be NULL or absent).
int check_ptrs(const char* fn, const char* name, const void* const* p, int n, bool needed)
{
    if (!p) return needed ? fail(RTP_EINVAL, "%s: NULL %s", fn, name) : RTP_OK;
    for (int i = 0; i < n; ++i) {
        if (needed && !p[i]) return fail(RTP_EINVAL, "%s: NULL %s for rank %d", fn, name, i);
        if (!aligned16(p[i])) return fail(RTP_EINVAL, "%s: %s of rank %d must be 16-byte aligned", fn, name, i);
    }
    return RTP_OK;
}

template <class T>
const void* const* cptr(T* const* p) { return reinterpret_cast<const void* const*>(p); }

size_t dsize(int dtype) { return dtype == RTP_F32 ? 4 : 2; }

int zero(const char* fn, void* const* p, int n, int64_t bytes, cudaStream_t s)
{
    for (int i = 0; p && i < n; ++i)
        if (cudaMemsetAsync(p[i], 0, (size_t)bytes, s) != cudaSuccess) return fail(RTP_ECUDA, "%s: cudaMemsetAsync failed", fn);
    return RTP_OK;
}

struct LinShape {
    bool row;
    int outs, ins;   // output and input buffers
    int64_t Kp, Np;  // a rank's weight [Kp, Np]
};

int linear_shape(const char* fn, int split, int P, int64_t M, int64_t K, int64_t N, int act, LinShape* s)
{
    if (split != RTP_SPLIT_COLUMN && split != RTP_SPLIT_ROW) return fail(RTP_EINVAL, "%s: unknown split %d", fn, split);
    TRY(check_common(fn, P, M, K, N, act));
    s->row = split == RTP_SPLIT_ROW;
    s->outs = s->row ? 1 : P;
    s->ins = s->row ? P : 1;
    const int64_t cut = s->row ? K : N;
    if (cut % P) return fail(RTP_ESHAPE, "%s: %s=%lld is not divisible by P=%d", fn, s->row ? "K" : "N", (long long)cut, P);
    s->Kp = s->row ? K / P : K;
    s->Np = s->row ? N : N / P;
    if (s->Kp % 8 || s->Np % 8)
        return fail(RTP_ESHAPE, "%s: a rank's weight extents %lld and %lld must be multiples of 8 (16-byte rows)", fn,
                    (long long)s->Kp, (long long)s->Np);
    return RTP_OK;
}

int linear_impl(const char* fn, int split, int P, int64_t M, int64_t K, int64_t N, const void* const* X,
                const void* const* W, const void* const* bias, const void* const* residual, int act, int out_dtype,
                void* const* H, void* const* out, rtp_stream stream)
{
    LinShape s;
    TRY(linear_shape(fn, split, P, M, K, N, act, &s));
    TRY(check_dtype(fn, "out", out_dtype));
    TRY(check_ptrs(fn, "weight", W, P, true));
    TRY(check_ptrs(fn, "bias", bias, s.outs, bias != nullptr));
    const bool some = M > 0;  // buffers of M rows may be NULL when M == 0
    TRY(check_ptrs(fn, "X", X, s.ins, some));
    TRY(check_ptrs(fn, "residual", residual, s.outs, some && residual));
    TRY(check_ptrs(fn, "H", cptr(H), s.outs, some && H));
    TRY(check_ptrs(fn, "out", cptr(out), s.outs, some));
    if (!some) return RTP_OK;
    LinGemm g;
    g.groups = P;
    g.fused = s.row;
    g.a_shared = !s.row;
    g.out_f32 = out_dtype == RTP_F32;
    g.act = act;
    g.rows = M;
    g.cols = s.Np;
    g.kdim = s.Kp;
    for (int i = 0; i < P; ++i) {
        g.A[i] = X[s.row ? i : 0];
        g.B[i] = W[i];
    }
    for (int i = 0; i < s.outs; ++i) {
        g.out[i] = out[i];
        if (H) g.out2[i] = H[i];
        if (bias) g.bias[i] = bias[i];
        if (residual) g.residual[i] = residual[i];
    }
    return forward(fn, g, false, static_cast<cudaStream_t>(stream));
}

int linear_backward_impl(const char* fn, int split, int P, int64_t M, int64_t K, int64_t N, const void* const* X,
                         const void* const* W, const void* const* H, const void* const* dout, int act, void* const* dH,
                         int dx_dtype, void* const* dX, int dw_dtype, void* const* dW, float* const* db,
                         rtp_stream stream_)
{
    LinShape s;
    TRY(linear_shape(fn, split, P, M, K, N, act, &s));
    TRY(check_dtype(fn, "dX", dx_dtype));
    TRY(check_dtype(fn, "dW", dw_dtype));
    const bool some = M > 0, has_act = act != RTP_ACT_NONE;
    TRY(check_ptrs(fn, "X", X, s.ins, some && dW));
    TRY(check_ptrs(fn, "weight", W, P, dX != nullptr));
    TRY(check_ptrs(fn, "H", H, s.outs, some && has_act));
    TRY(check_ptrs(fn, "dOut", dout, s.outs, some));
    TRY(check_ptrs(fn, "dH", cptr(dH), s.outs, some && has_act));
    TRY(check_ptrs(fn, "dX", cptr(dX), s.ins, some && dX));
    TRY(check_ptrs(fn, "dW", cptr(dW), P, dW != nullptr));
    TRY(check_ptrs(fn, "db", cptr(db), s.outs, db != nullptr));
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (!some) {  // no tokens: the weight and bias gradients are zero, dX is empty
        TRY(zero(fn, dW, P, s.Kp * s.Np * (int64_t)dsize(dw_dtype), stream));
        return zero(fn, reinterpret_cast<void* const*>(db), s.outs, s.Np * 4, stream);
    }
    if (has_act || db) {
        SumArgs a = {};
        for (int i = 0; i < s.outs; ++i) {
            a.dout[i] = static_cast<const __nv_bfloat16*>(dout[i]);
            if (has_act) {
                a.h[i] = static_cast<const __nv_bfloat16*>(H[i]);
                a.dh[i] = static_cast<__nv_bfloat16*>(dH[i]);
            }
            if (db) a.db[i] = db[i];
        }
        a.rows = M;
        a.cols = (int)s.Np;
        a.act = act;
        TRY(launch_act_grad(fn, a, s.outs, stream));
    }
    const void* const* d = has_act ? cptr(dH) : dout;
    if (dX) {  // column: sum_i dH_i W_i^T in one accumulator; row: dX_i = dH W_i^T
        LinGemm g;
        g.groups = P;
        g.fused = !s.row;
        g.a_shared = s.row;
        g.b_t = true;
        g.out_f32 = dx_dtype == RTP_F32;
        g.rows = M;
        g.cols = s.Kp;
        g.kdim = s.Np;
        for (int i = 0; i < P; ++i) {
            g.A[i] = d[s.row ? 0 : i];
            g.B[i] = W[i];
        }
        for (int i = 0; i < s.ins; ++i) g.out[i] = dX[i];
        TRY(launch_linear_gemm(fn, g, stream));
    }
    if (dW) {  // dW_i = X^T dH_i, or X_i^T dH
        LinGemm g;
        g.groups = P;
        g.a_t = true;
        g.a_shared = !s.row;
        g.out_f32 = dw_dtype == RTP_F32;
        g.rows = s.Kp;
        g.cols = s.Np;
        g.kdim = M;
        for (int i = 0; i < P; ++i) {
            g.A[i] = X[s.row ? i : 0];
            g.B[i] = d[s.row ? 0 : i];
            g.out[i] = dW[i];
        }
        TRY(launch_linear_gemm(fn, g, stream));
    }
    return RTP_OK;
}

int check_glu(const char* fn, int P, int64_t M, int64_t K, int64_t F, int64_t N, int act)
{
    TRY(check_common(fn, P, M, K, N, act));
    if (F < 1 || F % P) return fail(RTP_ESHAPE, "%s: F=%lld is not a positive multiple of P=%d", fn, (long long)F, P);
    const int64_t Fp = F / P;
    if (K % 8 || Fp % 8 || N % 8) return fail(RTP_ESHAPE, "%s: K, F/P and N must be multiples of 8 (16-byte rows)", fn);
    if (Fp >= (int64_t)1 << 31) return fail(RTP_ESHAPE, "%s: extents must stay below 2^31", fn);
    return RTP_OK;
}

int glu_impl(const char* fn, int P, int64_t M, int64_t K, int64_t F, int64_t N, const void* X, const void* const* Ag,
             const void* const* Au, const void* const* B, const void* residual, int act, void* const* Y, bool keep,
             void* const* Hg, void* const* Hu, int out_dtype, void* Z, rtp_stream stream_)
{
    TRY(check_glu(fn, P, M, K, F, N, act));
    TRY(check_dtype(fn, "Z", out_dtype));
    const bool some = M > 0;
    TRY(check_ptrs(fn, "gate weight", Ag, P, true));
    TRY(check_ptrs(fn, "up weight", Au, P, true));
    TRY(check_ptrs(fn, "B", B, P, true));
    TRY(check_ptrs(fn, "Y", cptr(Y), P, some));
    TRY(check_ptrs(fn, "Hg", cptr(Hg), P, some && keep));
    TRY(check_ptrs(fn, "Hu", cptr(Hu), P, some && keep));
    const void* whole[3] = {X, Z, residual};
    TRY(check_ptrs(fn, "X or Z", whole, 2, some));
    TRY(check_ptrs(fn, "residual", whole + 2, 1, false));
    if (!some) return RTP_OK;
    const int64_t Fp = F / P;
    LinGemm g1, g2;
    g1.epi = LIN_GLU;
    g1.groups = g2.groups = P;
    g1.a_shared = true;
    g2.fused = true;
    g1.act = act;
    g1.rows = g2.rows = M;
    g1.kdim = K;
    g1.cols = g2.kdim = Fp;
    g2.cols = N;
    g2.out_f32 = out_dtype == RTP_F32;
    for (int i = 0; i < P; ++i) {
        g1.A[i] = X;
        g1.B[i] = Ag[i];
        g1.B2[i] = Au[i];
        g1.out[i] = Y[i];
        if (keep) {
            g1.out2[i] = Hg[i];
            g1.out3[i] = Hu[i];
        }
        g2.A[i] = Y[i];
        g2.B[i] = B[i];
    }
    g2.out[0] = Z;
    g2.residual[0] = residual;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    TRY(forward(fn, g1, false, stream));
    // g1's kernels wait for their predecessors and do not write B, so B is ready
    return forward(fn, g2, true, stream);
}

int glu_backward_impl(const char* fn, int P, int64_t M, int64_t K, int64_t F, int64_t N, const void* X,
                      const void* const* Ag, const void* const* Au, const void* const* B, const void* const* Hg,
                      const void* const* Hu, const void* const* Y, const void* dZ, int act, void* const* dHg,
                      void* const* dHu, int dx_dtype, void* dX, int dw_dtype, void* const* dAg, void* const* dAu,
                      void* const* dB, rtp_stream stream_)
{
    TRY(check_glu(fn, P, M, K, F, N, act));
    TRY(check_dtype(fn, "dX", dx_dtype));
    TRY(check_dtype(fn, "the weight gradients", dw_dtype));
    const bool some = M > 0;
    const int64_t Fp = F / P;
    if ((dAg != nullptr) != (dAu != nullptr)) return fail(RTP_EINVAL, "%s: dAg and dAu come together", fn);
    TRY(check_ptrs(fn, "gate weight", Ag, P, dX != nullptr));
    TRY(check_ptrs(fn, "up weight", Au, P, dX != nullptr));
    TRY(check_ptrs(fn, "B", B, P, true));
    TRY(check_ptrs(fn, "Hg", Hg, P, some));
    TRY(check_ptrs(fn, "Hu", Hu, P, some));
    TRY(check_ptrs(fn, "Y", Y, P, some && dB));
    TRY(check_ptrs(fn, "dHg", cptr(dHg), P, some));
    TRY(check_ptrs(fn, "dHu", cptr(dHu), P, some));
    const void* whole[3] = {dZ, X, dX};
    TRY(check_ptrs(fn, "dZ", whole, 1, some));
    TRY(check_ptrs(fn, "X", whole + 1, 1, some && dAg));
    TRY(check_ptrs(fn, "dX", whole + 2, 1, false));
    TRY(check_ptrs(fn, "dAg", cptr(dAg), P, dAg != nullptr));
    TRY(check_ptrs(fn, "dAu", cptr(dAu), P, dAu != nullptr));
    TRY(check_ptrs(fn, "dB", cptr(dB), P, dB != nullptr));
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (!some) {  // no tokens: the weight gradients are zero, dX is empty
        const int64_t es = (int64_t)dsize(dw_dtype);
        TRY(zero(fn, dAg, P, K * Fp * es, stream));
        TRY(zero(fn, dAu, P, K * Fp * es, stream));
        return zero(fn, dB, P, Fp * N * es, stream);
    }
    if (dX || dAg) {  // dHg, dHu from dY = dZ B^T, which is not stored
        LinGemm g;
        g.epi = LIN_DGLU;
        g.groups = P;
        g.a_shared = true;
        g.b_t = true;
        g.act = act;
        g.rows = M;
        g.cols = Fp;
        g.kdim = N;
        for (int i = 0; i < P; ++i) {
            g.A[i] = dZ;
            g.B[i] = B[i];
            g.aux[i] = Hg[i];
            g.aux2[i] = Hu[i];
            g.out[i] = dHg[i];
            g.out2[i] = dHu[i];
        }
        TRY(launch_linear_gemm(fn, g, stream));
    }
    if (dX) {  // one accumulator over the gate and up products of every rank
        LinGemm g;
        g.groups = 2 * P;
        g.fused = true;
        g.b_t = true;
        g.out_f32 = dx_dtype == RTP_F32;
        g.rows = M;
        g.cols = K;
        g.kdim = Fp;
        for (int i = 0; i < P; ++i) {
            g.A[2 * i] = dHg[i];
            g.B[2 * i] = Ag[i];
            g.A[2 * i + 1] = dHu[i];
            g.B[2 * i + 1] = Au[i];
        }
        g.out[0] = dX;
        TRY(launch_linear_gemm(fn, g, stream));
    }
    if (dAg) {
        LinGemm g;
        g.groups = 2 * P;
        g.a_t = true;
        g.a_shared = true;
        g.out_f32 = dw_dtype == RTP_F32;
        g.rows = K;
        g.cols = Fp;
        g.kdim = M;
        for (int i = 0; i < P; ++i) {
            g.A[2 * i] = g.A[2 * i + 1] = X;
            g.B[2 * i] = dHg[i];
            g.B[2 * i + 1] = dHu[i];
            g.out[2 * i] = dAg[i];
            g.out[2 * i + 1] = dAu[i];
        }
        TRY(launch_linear_gemm(fn, g, stream));
    }
    if (dB) {
        LinGemm g;
        g.groups = P;
        g.a_t = true;
        g.out_f32 = dw_dtype == RTP_F32;
        g.rows = Fp;
        g.cols = N;
        g.kdim = M;
        for (int i = 0; i < P; ++i) {
            g.A[i] = Y[i];
            g.B[i] = dZ;
            g.out[i] = dB[i];
        }
        TRY(launch_linear_gemm(fn, g, stream));
    }
    return RTP_OK;
}

}  // namespace

}  // namespace rtp

using namespace rtp;

extern "C" {

int rtp_tp_linear(int split, int P, int64_t M, int64_t K, int64_t N, const void* const* X, const void* const* W_shards,
                  const void* const* bias, const void* const* residual, int act, rtp_dtype out_dtype, void* const* H,
                  void* const* out, rtp_stream stream)
{
    const char* fn = "rtp_tp_linear";
    return guarded(fn, [&] {
        return linear_impl(fn, split, P, M, K, N, X, W_shards, bias, residual, act, out_dtype, H, out, stream);
    });
}

int rtp_tp_linear_backward(int split, int P, int64_t M, int64_t K, int64_t N, const void* const* X,
                           const void* const* W_shards, const void* const* H, const void* const* dOut, int act,
                           void* const* dH, rtp_dtype dx_dtype, void* const* dX, rtp_dtype dw_dtype, void* const* dW,
                           float* const* db, rtp_stream stream)
{
    const char* fn = "rtp_tp_linear_backward";
    return guarded(fn, [&] {
        return linear_backward_impl(fn, split, P, M, K, N, X, W_shards, H, dOut, act, dH, dx_dtype, dX, dw_dtype, dW, db,
                                    stream);
    });
}

int rtp_tp_glu(int P, int64_t M, int64_t K, int64_t F, int64_t N, const void* X, const void* const* Ag_shards,
               const void* const* Au_shards, const void* const* B_shards, const void* residual, int act, void* const* Y,
               rtp_dtype out_dtype, void* Z, rtp_stream stream)
{
    const char* fn = "rtp_tp_glu";
    return guarded(fn, [&] {
        return glu_impl(fn, P, M, K, F, N, X, Ag_shards, Au_shards, B_shards, residual, act, Y, false, nullptr, nullptr,
                        out_dtype, Z, stream);
    });
}

int rtp_tp_glu_train_forward(int P, int64_t M, int64_t K, int64_t F, int64_t N, const void* X,
                             const void* const* Ag_shards, const void* const* Au_shards, const void* const* B_shards,
                             const void* residual, int act, void* const* Y, void* const* Hg, void* const* Hu,
                             rtp_dtype out_dtype, void* Z, rtp_stream stream)
{
    const char* fn = "rtp_tp_glu_train_forward";
    return guarded(fn, [&] {
        return glu_impl(fn, P, M, K, F, N, X, Ag_shards, Au_shards, B_shards, residual, act, Y, true, Hg, Hu, out_dtype, Z,
                        stream);
    });
}

int rtp_tp_glu_backward(int P, int64_t M, int64_t K, int64_t F, int64_t N, const void* X, const void* const* Ag_shards,
                        const void* const* Au_shards, const void* const* B_shards, const void* const* Hg,
                        const void* const* Hu, const void* const* Y, const void* dZ, int act, void* const* dHg,
                        void* const* dHu, rtp_dtype dx_dtype, void* dX, rtp_dtype dw_dtype, void* const* dAg,
                        void* const* dAu, void* const* dB, rtp_stream stream)
{
    const char* fn = "rtp_tp_glu_backward";
    return guarded(fn, [&] {
        return glu_backward_impl(fn, P, M, K, F, N, X, Ag_shards, Au_shards, B_shards, Hg, Hu, Y, dZ, act, dHg, dHu,
                                 dx_dtype, dX, dw_dtype, dAg, dAu, dB, stream);
    });
}

int rtp_product_launches(int32_t* counts)
{
    if (!counts) return fail(RTP_EINVAL, "rtp_product_launches: NULL argument");
    for (int i = 0; i < RTP_PRODUCT_FORMS; ++i) {
        counts[i] = product_launches[i];
        product_launches[i] = 0;
    }
    return RTP_OK;
}

}  // extern "C"
