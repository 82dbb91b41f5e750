// The same products for few rows (a token or a small batch being decoded), computed
// transposed, out^T = B^T A^T: 128 output columns ("features") of a CTA are the M
// operand of the MMA, the rows ("tokens"), up to 128 in steps of 16, its N operand.
// For LIN_GLU a CTA's 128 features are 64 gate and the same 64 up columns.
// LIN_LSE and LIN_EXP leave softmax statistics of 128 columns (softmax.cuh).
//
// With few tokens every weight is used a handful of times, so the weights' bytes
// over the HBM rate bound the time, and the tiles of the pair kernel would leave
// most of their rows, and with few columns most SMs, idle. Weights are used straight
// from their row-major form (an M-major operand). The K range (all ranks' K ranges
// when the ranks are summed) is cut into `split` parts over a cluster of CTAs: each
// part's float32 partial tile goes to its CTA's shared memory, and the CTAs then add
// up slices of it over distributed shared memory in the order of the parts, so the
// result does not depend on timing and no workspace is needed. Two CTAs fit on an
// SM, so that about 190 KB of loads are in flight on it.
// Measured: the gated 4096 x 16384 x 4096 block on 8 ranks, 1 row 64.5 us (its 403 MB of
// weights at 6250 GB/s), 128 rows 76; a row-parallel 16384 x 4096, 5 rows, 24.1 us.
#include <atomic>
#include <cstring>

#include "activation.cuh"
#include "linear.h"
#include "softmax.cuh"
#include "tcgen05.cuh"

namespace rtp {

namespace {

constexpr int FEAT = LIN_FEW_COLS;             // features of a CTA's tile
constexpr uint32_t SUB = 64 * BK * 2;          // one 64 x 64 box, 8 KB
constexpr uint32_t W_BYTES = FEAT * BK * 2;    // 16 KB
constexpr int THREADS = 256;                   // warps w and w + 4 read the same quarter of the tensor memory's lanes
constexpr int MAX_STAGES = 8;
constexpr int MAX_SPLIT = 8;                   // portable cluster size
constexpr size_t SMEM_LIMIT = 113 * 1024;      // per CTA, two on an SM (228 KB, 1 KB reserved per CTA)
constexpr size_t SMEM_EXTRA = 1024 + 256;      // alignment; barriers

struct Args {
    CUtensorMap tw[LIN_MAX_GROUPS];  // B operands; LIN_GLU: [g] gate, [LIN_MAX_RANKS + g] up
    CUtensorMap tx[LIN_MAX_RANKS];   // A operands
    void* out[LIN_MAX_RANKS];
    __nv_bfloat16* out2[LIN_MAX_RANKS];
    __nv_bfloat16* out3[LIN_MAX_RANKS];
    const __nv_bfloat16* bias[LIN_MAX_RANKS];
    const __nv_bfloat16* residual[LIN_MAX_RANKS];
    int32_t fused, kb_per_group, kbs;
    int32_t tiles;  // feature tiles of a group
    int32_t rows, cols, ntok, tmem_cols;
    int32_t split, stages;
    int32_t act, keep, weights_ready;
    unsigned long long wait_ns;  // limit of a wait for this kernel's own progress
    SoftmaxArgs softmax;
    int64_t ldo;  // LIN_EXP: row stride of out
};

__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ float4 bf16x4(const __nv_bfloat16* p)
{
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
__device__ __forceinline__ void store_bf16x4(__nv_bfloat16* p, float4 v)
{
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }
__device__ __forceinline__ float4 mul4(float4 a, float4 b) { return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w); }

template <int EPI, bool F32>
__global__ void __launch_bounds__(THREADS, 2) linear_few_kernel(const __grid_constant__ Args a)
{
    constexpr int CTA_COLS = EPI == LIN_GLU ? FEAT / 2 : FEAT;  // output columns of a CTA
    extern __shared__ uint8_t smem_raw[];
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t stage_bytes = W_BYTES + (uint32_t)a.ntok * (BK * 2);
    const uint32_t bar0 = smem + (uint32_t)a.stages * stage_bytes;
    auto full_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(MAX_STAGES + s); };
    const uint32_t acc_bar = bar0 + 8u * (uint32_t)(2 * MAX_STAGES), drain_bar = acc_bar + 8u;
    volatile uint32_t* tmem_slot =
        reinterpret_cast<volatile uint32_t*>(smem_raw + (bar0 - smem_u32(smem_raw)) + 8u * (2 * MAX_STAGES + 2));
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = (int)cluster_rank();  // K part
    const int tile = (int)blockIdx.x / a.split, g = tile / a.tiles, f0 = (tile - g * a.tiles) * CTA_COLS;
    const int kb0 = (int)((int64_t)a.kbs * part / a.split), kb1 = (int)((int64_t)a.kbs * (part + 1) / a.split);
    const int n = kb1 - kb0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(acc_bar, 1);
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {  // the descriptors this CTA will use, one a lane
        const int kg = a.fused ? kb0 / a.kb_per_group + lane : g;
        if (a.fused ? kg <= (kb1 - 1) / a.kb_per_group : lane == 0) {
            prefetch_map(&a.tw[kg]);
            prefetch_map(&a.tx[kg]);
            if (EPI == LIN_GLU) prefetch_map(&a.tw[LIN_MAX_RANKS + kg]);
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32((const void*)tmem_slot)),
                     "r"(a.tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            auto load_w = [&](int i, int s) {
                const int kb = kb0 + i, kg = a.fused ? kb / a.kb_per_group : 0;
                const int k = (kb - kg * a.kb_per_group) * BK, wg = a.fused ? kg : g;
                const uint32_t dst = smem + (uint32_t)s * stage_bytes;
                if constexpr (EPI == LIN_GLU) {
                    tma_load_2d(dst, &a.tw[wg], full_bar(s), f0, k);
                    tma_load_2d(dst + SUB, &a.tw[LIN_MAX_RANKS + wg], full_bar(s), f0, k);
                } else {
                    tma_load_2d(dst, &a.tw[wg], full_bar(s), f0, k);
                    tma_load_2d(dst + SUB, &a.tw[wg], full_bar(s), f0 + 64, k);
                }
            };
            auto load_x = [&](int i, int s) {
                const int kb = kb0 + i, kg = a.fused ? kb / a.kb_per_group : 0;
                tma_load_2d(smem + (uint32_t)s * stage_bytes + W_BYTES, &a.tx[a.fused ? kg : g], full_bar(s),
                            (kb - kg * a.kb_per_group) * BK, 0);
            };
            // Weights that nothing on the stream can still be writing are fetched
            // while the previous kernel finishes.
            const int early = a.weights_ready ? min(n, a.stages) : 0;
            for (int i = 0; i < early; ++i) {
                mbar_expect_tx(full_bar(i), stage_bytes);
                load_w(i, i);
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
            // This kernel's own dependents may be set up from here on: whatever
            // ran before this kernel is complete.
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            for (int i = 0; i < early; ++i) load_x(i, i);
            int s = early == a.stages ? 0 : early;
            uint32_t phase = early == a.stages ? 1u : 0u;
            int issued = early;
            for (int i = early; i < n; ++i) {
                if (!wait_bar(empty_bar(s), phase ^ 1u, abort_flag, ERR_PRODUCER, a.wait_ns)) break;
                mbar_expect_tx(full_bar(s), stage_bytes);
                load_w(i, s);
                load_x(i, s);
                ++issued;
                if (++s == a.stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (issued < n)  // gave up: the loads in flight land before the CTA leaves
                for (int i = max(0, issued - a.stages); i < issued; ++i)
                    drain_wait(full_bar(i % a.stages), (uint32_t)((i / a.stages) & 1));
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | ((uint32_t)(a.ntok >> 3) << 17) |
                                   ((uint32_t)(FEAT >> 4) << 24);
            // weights M-major: 2048-byte steps (16 K rows), the two 64-wide boxes SUB
            // bytes apart; tokens K-major: 32-byte steps (16 bf16) in the 128-byte
            // swizzle row, 8-row groups 1024 bytes apart
            const uint64_t desc_w = smem_desc(smem, SUB, 1024u), desc_x = smem_desc(smem + W_BYTES, 16u, 1024u);
            int s = 0;
            uint32_t phase = 0;
            bool ok = true;
            // The rows are fetched once the previous kernel is complete, so nothing is
            // lost by waiting for it here too, and the limit of the waits below then
            // covers this kernel's progress, not that kernel's run time.
            asm volatile("griddepcontrol.wait;" ::: "memory");
            for (int i = 0; i < n; ++i) {
                if (!wait_bar(full_bar(s), phase, abort_flag, ERR_MMA_STAGE, a.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t off = (uint64_t)((uint32_t)s * stage_bytes >> 4);
#pragma unroll
                for (int k = 0; k < BK / 16; ++k)
                    mma_bf16(tmem_base, desc_w + off + (uint64_t)(2048u * k >> 4), desc_x + off + (uint64_t)(32u * k >> 4),
                             idesc, (i > 0 || k > 0) ? 1u : 0u);
                mma_commit(empty_bar(s));
                if (++s == a.stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (ok) {
                mma_commit(acc_bar);
            } else {
                mma_commit(drain_bar);
                drain_wait(drain_bar, 0);
            }
        }
        __syncwarp();
    }

    // ---------------- the partial tile to shared memory, then the sum ----------------
    // Every load has landed and every MMA is done when acc_bar completes, so the
    // ring's memory is free: token t, feature f at float t * 128 + f.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // A thread takes 4 neighbouring output columns of one token, UNROLL such quads
    // at a time: the loads of the other operands, then of the partials, of all of
    // them are in flight together (one by one, each cost its full latency: the
    // epilogue of 256 tokens took 50 us). The first quads' other operands are
    // fetched while the product runs.
    constexpr int QUADS = CTA_COLS / 4, UNROLL = 4;
    const int step = a.split * THREADS, items = a.rows * QUADS;
    float4 u[UNROLL], x[UNROLL];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int j = 0; j < UNROLL; ++j) {
            const int i = i0 + j * step, t = i / QUADS, f = (i - t * QUADS) * 4;
            u[j] = x[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if constexpr (EPI == LIN_OUT) {
                if (i >= items || f0 + f >= a.cols) continue;
                if (a.bias[g]) u[j] = bf16x4(a.bias[g] + f0 + f);
                if (a.residual[g]) x[j] = bf16x4(a.residual[g] + (int64_t)t * a.cols + f0 + f);
            }
        }
    };
    int i0 = part * THREADS + (int)threadIdx.x;
    fetch(i0);
    int ok = 1;
    if (lane == 0) ok = wait_bar(acc_bar, 0, abort_flag, ERR_EPILOGUE, a.wait_ns) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    tc_fence_after();
    if (ok) {
        const int quarter = warp & 3;
        const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16);
        for (int c = 16 * (warp >> 2); c < a.rows; c += 16 * (THREADS / 128)) {
            uint32_t r[16];
            tmem_ld_16cols(taddr + (uint32_t)c, r);
            tmem_ld_wait(r);
            const uint32_t dst = smem + 4u * (uint32_t)(c * FEAT + quarter * 32 + lane);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + 4u * FEAT * j), "r"(r[j]) : "memory");
        }
    }
    tc_fence_before();
    if (a.split > 1) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(a.tmem_cols) : "memory");
    auto sum4 = [&](int t, int f) {
        const uint32_t addr = smem + 4u * (uint32_t)(t * FEAT + f);
        if (a.split == 1) return ld_shared_f4(addr);
        float4 v = ld_cluster_f4(map_to_rank(addr, 0));
        for (int r = 1; r < a.split; ++r) v = add4(v, ld_cluster_f4(map_to_rank(addr, (uint32_t)r)));
        return v;
    };
    if constexpr (EPI == LIN_LSE || EPI == LIN_EXP) {
        // A warp takes a token at a time, a lane 4 of its 128 features.
        const int f = 4 * lane, cols = min(FEAT, a.cols - f0);
        const int64_t first = (int64_t)g * a.cols + f0;
        const int valid = min(valid_columns(a.softmax, first, FEAT), cols);
#pragma unroll 2
        for (int t = part * (THREADS / 32) + warp; t < a.rows; t += a.split * (THREADS / 32)) {
            const float4 w = sum4(t, f);
            float v[4] = {w.x, w.y, w.z, w.w}, e[4], ref = 0.0f, sum;
            const int target = target_in(a.softmax, t, first, valid) - f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (f + j >= valid) v[j] = minus_infinity();
                if (target == j) a.softmax.target_logit[t] = v[j];
            }
            auto terms = [&]() {
                sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) sum += e[j] = exp2_fast(fmaf(v[j], LOG2E, -ref));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            };
            terms();
            if (valid > 0 && !in_range(sum)) {
                float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                ref = finite_ref(top * LOG2E);
                terms();
            }
            if (sum == 0.0f) ref = minus_infinity();
            if (lane == 0) a.softmax.stats[(int64_t)t * a.softmax.parts + tile] = make_float2(ref, sum);
            if (EPI == LIN_EXP && f < cols)
                store_bf16x4(static_cast<__nv_bfloat16*>(a.out[g]) + (int64_t)t * a.ldo + f0 + f,
                             takes_part(a.softmax, t) ? make_float4(e[0], e[1], e[2], e[3]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        }
    }
    while (EPI != LIN_LSE && EPI != LIN_EXP && i0 < items) {
        float4 v[UNROLL];
#pragma unroll
        for (int j = 0; j < UNROLL; ++j) {
            const int i = i0 + j * step, t = i / QUADS, f = (i - t * QUADS) * 4;
            v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i >= items || f0 + f >= a.cols) continue;
            v[j] = sum4(t, f);
            if constexpr (EPI == LIN_GLU) u[j] = sum4(t, 64 + f);
        }
#pragma unroll
        for (int j = 0; j < UNROLL; ++j) {
            const int i = i0 + j * step, t = i / QUADS, f = (i - t * QUADS) * 4;
            if (i >= items || f0 + f >= a.cols) continue;
            const int64_t at = (int64_t)t * a.cols + f0 + f;
            if constexpr (EPI == LIN_GLU) {
                if (a.keep) {
                    store_bf16x4(a.out2[g] + at, v[j]);
                    store_bf16x4(a.out3[g] + at, u[j]);
                }
            } else {
                v[j] = add4(v[j], u[j]);
                if (a.keep) store_bf16x4(a.out2[g] + at, v[j]);
            }
            with_act(a.act, [&](auto tag) {
                constexpr int ACT = decltype(tag)::value;
                v[j] = make_float4(act_value<ACT, F32>(v[j].x), act_value<ACT, F32>(v[j].y), act_value<ACT, F32>(v[j].z),
                                   act_value<ACT, F32>(v[j].w));
            });
            v[j] = EPI == LIN_GLU ? mul4(v[j], u[j]) : add4(v[j], x[j]);
            if constexpr (F32) *reinterpret_cast<float4*>(static_cast<float*>(a.out[g]) + at) = v[j];
            else store_bf16x4(static_cast<__nv_bfloat16*>(a.out[g]) + at, v[j]);
        }
        i0 += UNROLL * step;
        if (i0 < items) fetch(i0);
    }
    // No CTA leaves while a peer may still read its partial.
    if (a.split > 1) cluster_sync();
}

// ---- host side --------------------------------------------------------------------

template <int EPI, bool F32>
int launch_t(const char* fn, const Args& args, unsigned tiles, size_t smem, cudaStream_t stream)
{
    static std::atomic<bool> ready[64];
    auto kernel = linear_few_kernel<EPI, F32>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return fail(RTP_ECUDA, "%s: no CUDA device", fn);
    if (!ready[dev].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_LIMIT);
        if (e != cudaSuccess) return fail(RTP_ECUDA, "%s: cudaFuncSetAttribute: %s", fn, cudaGetErrorString(e));
        ready[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)args.split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(tiles * (unsigned)args.split);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args);
    if (e != cudaSuccess) return fail(RTP_ECUDA, "%s: few-row launch failed: %s", fn, cudaGetErrorString(e));
    ++product_launches[RTP_PRODUCT_FEW];
    return RTP_OK;
}

}  // namespace

thread_local int32_t product_launches[RTP_PRODUCT_FORMS];

int device_sms(int* n)
{
    static std::atomic<int> sms[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return RTP_ECUDA;
    int v = sms[dev].load(std::memory_order_acquire);
    if (!v) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) return RTP_ECUDA;
        sms[dev].store(v, std::memory_order_release);
    }
    *n = v;
    return RTP_OK;
}

int launch_linear_few(const char* fn, const LinGemm& p, bool weights_ready, cudaStream_t stream)
{
    int st, sms = 0;
    if (device_sms(&sms)) return fail(RTP_ECUDA, "%s: no CUDA device", fn);
    static thread_local Args a;
    std::memset(&a, 0, sizeof a);
    const int cta_cols = p.epi == LIN_GLU ? FEAT / 2 : FEAT;
    a.ntok = (int)((p.rows + 15) / 16 * 16);
    for (a.tmem_cols = 32; a.tmem_cols < a.ntok;) a.tmem_cols *= 2;
    // The ring also holds a partial tile, 512 bytes a token: 64 KB at most, while the
    // smallest ring (96 tokens, 3 stages of 28 KB) has 84.
    const size_t stage = W_BYTES + (size_t)a.ntok * (BK * 2);
    a.stages = (int)((SMEM_LIMIT - SMEM_EXTRA) / stage);
    if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
    for (int g = 0; g < p.groups; ++g) {
        if ((st = make_map(&a.tw[g], p.B[g], p.kdim, p.cols, BK))) return st;
        if (p.epi == LIN_GLU && (st = make_map(&a.tw[LIN_MAX_RANKS + g], p.B2[g], p.kdim, p.cols, BK))) return st;
        if (g > 0 && p.A[g] == p.A[g - 1]) a.tx[g] = a.tx[g - 1];
        else if ((st = make_map(&a.tx[g], p.A[g], p.rows, p.kdim, a.ntok))) return st;
    }
    const int outs = p.fused ? 1 : p.groups;
    for (int g = 0; g < outs; ++g) {
        a.out[g] = p.out[g];
        a.out2[g] = static_cast<__nv_bfloat16*>(p.out2[g]);
        a.out3[g] = static_cast<__nv_bfloat16*>(p.out3[g]);
        a.bias[g] = static_cast<const __nv_bfloat16*>(p.bias[g]);
        a.residual[g] = static_cast<const __nv_bfloat16*>(p.residual[g]);
    }
    a.keep = p.out2[0] != nullptr;
    a.fused = p.fused;
    a.kb_per_group = (int)((p.kdim + BK - 1) / BK);
    a.kbs = (p.fused ? p.groups : 1) * a.kb_per_group;
    a.tiles = (int)((p.cols + cta_cols - 1) / cta_cols);
    a.rows = (int)p.rows;
    a.cols = (int)p.cols;
    a.act = p.act;
    a.softmax = softmax_args(p.softmax, outs * a.tiles);
    a.ldo = p.ldo ? p.ldo : p.cols;
    a.weights_ready = weights_ready;
    int64_t wait_ns = (int64_t)WAIT_LIMIT_NS;
    take_hook(RTP_HOOK_WAIT_LIMIT, &wait_ns);
    a.wait_ns = (unsigned long long)wait_ns;
    const int64_t tiles = (int64_t)outs * a.tiles;
    if (tiles * MAX_SPLIT >= ((int64_t)1 << 31)) return fail(RTP_ESHAPE, "%s: too many tiles", fn);
    // K parts: one CTA an SM as long as each has 4 K blocks, two an SM as long as each
    // has 8 (measured at 1 to 128 rows: 2048 x 2048 in 8 parts of 4 blocks 5.1 us, in 4
    // of 8 5.9; the gated 1024 x 4096 x 1024 block in parts of 4 blocks at two CTAs an
    // SM 14.0 us, of 8 blocks at one 12.8)
    a.split = 1;
    while (a.split < MAX_SPLIT && tiles * a.split * 2 <= 2 * sms &&
           a.kbs >= 2 * a.split * (tiles * a.split * 2 <= sms ? 4 : 8))
        a.split *= 2;
    const size_t smem = (size_t)a.stages * stage + SMEM_EXTRA;
    if (p.epi == LIN_LSE) return launch_t<LIN_LSE, false>(fn, a, (unsigned)tiles, smem, stream);
    if (p.epi == LIN_EXP) return launch_t<LIN_EXP, false>(fn, a, (unsigned)tiles, smem, stream);
    if (p.epi == LIN_GLU) return launch_t<LIN_GLU, false>(fn, a, (unsigned)tiles, smem, stream);
    return p.out_f32 ? launch_t<LIN_OUT, true>(fn, a, (unsigned)tiles, smem, stream)
                     : launch_t<LIN_OUT, false>(fn, a, (unsigned)tiles, smem, stream);
}

int take_linear_few_error(void* stream, uint32_t* code) { return take_tp_error(stream, code); }

}  // namespace rtp
