// Global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum over counted tensors and their elements of g^2)
//   c    = min(1, max_norm / (norm + 1e-6)),   g' = c g
//
// HBM bound. Two kernels: the first reads the counted gradients and leaves one
// float64 sum per block; the second sums those in a fixed order (every block for
// itself), and scales. Blocks and the chunks they take depend on the sizes and
// the device alone, so results are the same from run to run. The second kernel
// walks the chunks backwards: what the first one read last is still in L2.
//
// Squares are added in float32 over a thread's part of one chunk (at most 64
// values, still in its registers) and across chunks in float64. A part whose
// float32 sum is outside [2^-60, 2^100] is added again in float64, so that the
// norm neither overflows nor underflows where it is itself a float32 number
// (below 2^-60 a lost square would matter, above 2^100 the next could overflow).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <type_traits>
#include <vector>

#include "rtp_internal.h"

namespace rtp {

namespace {

constexpr int THREADS = 256;
constexpr int BLOCKS_PER_SM = 4;
constexpr int MAX_BLOCKS = 1216;        // partial sums of one launch
constexpr int STEP_BYTES = THREADS * 16;  // one 16-byte vector a thread

struct Item {
    const void* src;
    void* dst;
    int64_t numel;
    uint32_t chunk0;  // first chunk
    uint32_t dtype;
};
template <int N>
struct Table {
    Item items[N];
    int32_t n;
    uint32_t chunks;
};
constexpr int SMALL = 64, LARGE = 512;  // tensors of one launch (2 KB or 16 KB of parameters)

// Item of chunk c (uniform over the block): the last one whose chunk0 is <= c.
template <int N>
__device__ __forceinline__ int find_item(const Table<N>& t, uint32_t c)
{
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.items[mid].chunk0 <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <class Fn>
__device__ __forceinline__ void each(const uint4& v, bool bf16, Fn&& fn)
{
    if (bf16) {
        fn(lo_f(v.x)), fn(hi_f(v.x)), fn(lo_f(v.y)), fn(hi_f(v.y));
        fn(lo_f(v.z)), fn(hi_f(v.z)), fn(lo_f(v.w)), fn(hi_f(v.w));
    } else {
        fn(__uint_as_float(v.x)), fn(__uint_as_float(v.y)), fn(__uint_as_float(v.z)), fn(__uint_as_float(v.w));
    }
}

__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double warp_sum[THREADS / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) v += warp_sum[w];
    return v;
}

// A chunk is V vectors of 16 bytes a thread. Tensors whose address is not a
// multiple of 16 go element by element.
template <int V, int N>
__global__ void __launch_bounds__(THREADS) grad_norm_kernel(const __grid_constant__ Table<N> t, double* partials)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    double acc = 0.0;
    for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Item& it = t.items[find_item(t, c)];
        const bool bf16 = it.dtype == RTP_BF16;
        const int per = bf16 ? 8 : 4;  // elements of a vector
        const int64_t e0 = (int64_t)(c - it.chunk0) * (V * THREADS * per);
        const int64_t left = min(it.numel - e0, (int64_t)(V * THREADS * per));
        uint4 v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (((uintptr_t)it.src & 15u) == 0) {
            const int64_t vec0 = e0 / per;
            const int nvec = (int)(left / per), tail = (int)(left - (int64_t)nvec * per);
            const uint4* p = static_cast<const uint4*>(it.src) + vec0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int at = i * THREADS + (int)threadIdx.x;
                if (at < nvec) v[i] = __ldg(p + at);
            }
            if ((int)threadIdx.x < tail) {  // the elements after the last whole vector, one a thread
                const int64_t e = e0 + (int64_t)nvec * per + threadIdx.x;
                const float x = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(it.src)[e])
                                     : static_cast<const float*>(it.src)[e];
                acc += (double)x * (double)x;
            }
        } else {
            for (int e = threadIdx.x; e < (int)left; e += THREADS) {
                const float x = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(it.src)[e0 + e])
                                     : static_cast<const float*>(it.src)[e0 + e];
                acc += (double)x * (double)x;
            }
            continue;
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) each(v[i], bf16, [&](float x) { s += x * x; });
        if (s >= 0x1p-60f && s <= 0x1p100f) {
            acc += (double)s;
        } else {
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) any |= v[i].x | v[i].y | v[i].z | v[i].w;
            if (any & 0x7FFF7FFFu || (!bf16 && any & 0x7FFFFFFFu)) {
#pragma unroll
                for (int i = 0; i < V; ++i) each(v[i], bf16, [&](float x) { acc += (double)x * (double)x; });
            }
        }
    }
    const double total = block_sum(acc);
    if (threadIdx.x == 0) partials[blockIdx.x] = total;
}

__device__ __forceinline__ uint32_t scale2(uint32_t w, float c)
{
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(lo_f(w) * c)) |
           ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(hi_f(w) * c)) << 16);
}

template <int V, int N>
__global__ void __launch_bounds__(THREADS) grad_scale_kernel(const __grid_constant__ Table<N> t, const double* partials,
                                                             int n_partials, float max_norm, float* norm, int in_place)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    double s = 0.0;
    for (int i = threadIdx.x; i < n_partials; i += THREADS) s += __ldcg(partials + i);
    const float total = (float)sqrt(block_sum(s));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    float k = max_norm / (total + 1e-6f);
    if (k > 1.0f) k = 1.0f;  // a NaN stays one
    if (in_place && k == 1.0f) return;
    for (uint32_t b = blockIdx.x; b < t.chunks; b += gridDim.x) {
        const uint32_t c = t.chunks - 1 - b;
        const Item& it = t.items[find_item(t, c)];
        const bool bf16 = it.dtype == RTP_BF16;
        const int per = bf16 ? 8 : 4;
        const int64_t e0 = (int64_t)(c - it.chunk0) * (V * THREADS * per);
        const int64_t left = min(it.numel - e0, (int64_t)(V * THREADS * per));
        if ((((uintptr_t)it.src | (uintptr_t)it.dst) & 15u) == 0) {
            const int nvec = (int)(left / per), tail = (int)(left - (int64_t)nvec * per);
            const uint4* p = static_cast<const uint4*>(it.src) + e0 / per;
            uint4* q = static_cast<uint4*>(it.dst) + e0 / per;
            uint4 v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int at = i * THREADS + (int)threadIdx.x;
                if (at < nvec) v[i] = __ldcs(p + at);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int at = i * THREADS + (int)threadIdx.x;
                if (at >= nvec) break;
                uint4 w;
                if (bf16) w = make_uint4(scale2(v[i].x, k), scale2(v[i].y, k), scale2(v[i].z, k), scale2(v[i].w, k));
                else
                    w = make_uint4(__float_as_uint(__uint_as_float(v[i].x) * k), __float_as_uint(__uint_as_float(v[i].y) * k),
                                   __float_as_uint(__uint_as_float(v[i].z) * k), __float_as_uint(__uint_as_float(v[i].w) * k));
                __stcs(q + at, w);
            }
            if ((int)threadIdx.x < tail) {
                const int64_t e = e0 + (int64_t)nvec * per + threadIdx.x;
                if (bf16)
                    static_cast<__nv_bfloat16*>(it.dst)[e] =
                        __float2bfloat16_rn(__bfloat162float(static_cast<const __nv_bfloat16*>(it.src)[e]) * k);
                else static_cast<float*>(it.dst)[e] = static_cast<const float*>(it.src)[e] * k;
            }
        } else {
            for (int i = threadIdx.x; i < (int)left; i += THREADS) {
                const int64_t e = e0 + i;
                if (bf16)
                    static_cast<__nv_bfloat16*>(it.dst)[e] =
                        __float2bfloat16_rn(__bfloat162float(static_cast<const __nv_bfloat16*>(it.src)[e]) * k);
                else static_cast<float*>(it.dst)[e] = static_cast<const float*>(it.src)[e] * k;
            }
        }
    }
}

// ---- host side --------------------------------------------------------------------

int sm_count(const char* fn, int* n)
{
    static std::atomic<int> sms[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return fail(RTP_ECUDA, "%s: no CUDA device", fn);
    int v = sms[dev].load(std::memory_order_acquire);
    if (!v) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
            return fail(RTP_ECUDA, "%s: cudaDeviceGetAttribute failed", fn);
        sms[dev].store(v, std::memory_order_release);
    }
    *n = v;
    return RTP_OK;
}

size_t esize(int dtype) { return dtype == RTP_F32 ? 4 : 2; }

// The launches of one pass over `items` (chunk0 not yet set): call(table, blocks, index of launch).
template <int V, int N, class Call>
int each_launch(std::vector<Item>& items, int blocks, Call&& call)
{
    static thread_local Table<N> t;
    size_t i = 0;
    for (int launch = 0; i < items.size(); ++launch) {
        t.n = 0;
        uint64_t chunks = 0;
        for (; i < items.size() && t.n < N; ++i) {
            const uint64_t bytes = (uint64_t)items[i].numel * esize((int)items[i].dtype);
            const uint64_t add = (bytes + (uint64_t)V * STEP_BYTES - 1) / ((uint64_t)V * STEP_BYTES);
            if (t.n > 0 && chunks + add > 0x7fffffffu) break;
            items[i].chunk0 = (uint32_t)chunks;
            t.items[t.n++] = items[i];
            chunks += add;
        }
        t.chunks = (uint32_t)chunks;
        int st = call(t, (int)std::min<uint64_t>(chunks, (uint64_t)blocks), launch);
        if (st) return st;
    }
    return RTP_OK;
}

template <int V, int N>
int run(const char* fn, std::vector<Item>& counted, std::vector<Item>& all, double* partials, bool clip, float max_norm,
        bool in_place, float* norm, int blocks, cudaStream_t stream)
{
    int n_partials = 0;
    int st = each_launch<V, N>(counted, blocks, [&](const Table<N>& t, int grid, int) {
        grad_norm_kernel<V, N><<<grid, THREADS, 0, stream>>>(t, partials + n_partials);
        n_partials += grid;
        cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? RTP_OK : fail(RTP_ECUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
    });
    if (st) return st;
    auto scale = [&](const Table<N>& t, int grid, int launch) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        // The first launch follows the norm kernel and may be set up while that one
        // finishes. The later ones follow a kernel that does not announce dependents.
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3((unsigned)std::max(grid, 1));
        cfg.blockDim = dim3(THREADS);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = launch == 0 ? 1 : 0;
        cudaError_t e = cudaLaunchKernelEx(&cfg, grad_scale_kernel<V, N>, t, (const double*)partials, n_partials, max_norm,
                                           launch == 0 ? norm : (float*)nullptr, in_place ? 1 : 0);
        return e == cudaSuccess ? RTP_OK : fail(RTP_ECUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
    };
    if (!clip || all.empty()) {  // the norm alone
        static thread_local Table<N> none;
        none.n = 0;
        none.chunks = 0;
        return scale(none, 1, 0);
    }
    return each_launch<V, N>(all, blocks, scale);
}

// Launches of at most LARGE tensors; one more for each time 2^31 chunks are full
// (8 TB of gradients: never).
int64_t workspace_bytes(int n) { return (int64_t)((n + SMALL - 1) / SMALL + 1) * MAX_BLOCKS * 8; }

int norm_impl(const char* fn, int n, const int32_t* dtypes, const int64_t* numels, const void* const* grads,
              const uint8_t* counted, bool clip, float max_norm, void* const* out, void* workspace, float* norm,
              rtp_stream stream)
{
    if (n < 0) return fail(RTP_EINVAL, "%s: n = %d", fn, n);
    if (n > 0 && (!dtypes || !numels || !grads)) return fail(RTP_EINVAL, "%s: NULL argument", fn);
    if (!workspace || ((uintptr_t)workspace & 7u)) return fail(RTP_EINVAL, "%s: the workspace must be there and 8-byte aligned", fn);
    if (!norm || ((uintptr_t)norm & 3u)) return fail(RTP_EINVAL, "%s: norm must be there and 4-byte aligned", fn);
    if (clip && !(max_norm >= 0.0f)) return fail(RTP_EINVAL, "%s: max_norm %g is not a number >= 0", fn, (double)max_norm);
    std::vector<Item> in, all;
    struct Range {
        uintptr_t lo, hi;
        int i;
        bool dst;
    };
    std::vector<Range> ranges;
    uint64_t bytes = 0;
    for (int i = 0; i < n; ++i) {
        if (dtypes[i] != RTP_F32 && dtypes[i] != RTP_BF16) return fail(RTP_EINVAL, "%s: tensor %d is of unknown type %d", fn, i, dtypes[i]);
        if (numels[i] < 0 || numels[i] >= (int64_t)1 << 44) return fail(RTP_ESHAPE, "%s: tensor %d has %lld elements", fn, i, (long long)numels[i]);
        if (numels[i] == 0) continue;
        const size_t es = esize(dtypes[i]);
        void* dst = out ? out[i] : const_cast<void*>(grads[i]);
        if (!grads[i] || (clip && !dst)) return fail(RTP_EINVAL, "%s: NULL buffer of tensor %d", fn, i);
        if (((uintptr_t)grads[i] | (clip ? (uintptr_t)dst : 0)) & (es - 1))
            return fail(RTP_EINVAL, "%s: tensor %d is not aligned to its elements", fn, i);
        Item it = {grads[i], dst, numels[i], 0u, (uint32_t)dtypes[i]};
        all.push_back(it);
        if (!counted || counted[i]) in.push_back(it);
        bytes += (uint64_t)numels[i] * es;
        if (clip) {
            const uint64_t len = (uint64_t)numels[i] * es;
            if (dst != grads[i]) ranges.push_back(Range{(uintptr_t)grads[i], (uintptr_t)grads[i] + len, i, false});
            ranges.push_back(Range{(uintptr_t)dst, (uintptr_t)dst + len, i, true});
        }
    }
    // An output may be its own input (a tensor clipped in place), and shares bytes
    // with nothing else: the chunks are read and written in no fixed order, and a
    // tensor listed twice would be scaled twice.
    std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    const Range *src = nullptr, *dst = nullptr;  // the ranges of either kind that reach furthest so far
    for (const Range& r : ranges) {
        if ((dst && dst->hi > r.lo) || (r.dst && src && src->hi > r.lo))
            return fail(RTP_EINVAL, "%s: the output of tensor %d shares bytes with another buffer", fn, r.dst ? r.i : dst->i);
        const Range*& best = r.dst ? dst : src;
        if (!best || r.hi > best->hi) best = &r;
    }
    const bool in_place = clip && !out;
    int sms = 0, st;
    if ((st = sm_count(fn, &sms))) return st;
    const int blocks = std::min(sms * BLOCKS_PER_SM, MAX_BLOCKS);
    const uint64_t per_block = bytes / (uint64_t)blocks;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    double* ws = static_cast<double*>(workspace);
    auto go = [&](auto v) {
        constexpr int V = decltype(v)::value;
        if (all.size() <= SMALL) return run<V, SMALL>(fn, in, all, ws, clip, max_norm, in_place, norm, blocks, s);
        return run<V, LARGE>(fn, in, all, ws, clip, max_norm, in_place, norm, blocks, s);
    };
    // Chunks of 32 KB keep 8 loads in flight a thread; when there are too few of
    // them for every block, chunks of 4 KB spread the work over the SMs.
    if (per_block >= 8u * STEP_BYTES) return go(std::integral_constant<int, 8>());
    return go(std::integral_constant<int, 1>());
}

}  // namespace

}  // namespace rtp

using namespace rtp;

extern "C" {

int64_t rtp_grad_workspace_bytes(int n) { return n < 0 ? 0 : workspace_bytes(n); }

int rtp_grad_norm(int n, const int32_t* dtypes, const int64_t* numels, const void* const* grads, const uint8_t* counted,
                  void* workspace, float* norm, rtp_stream stream)
{
    const char* fn = "rtp_grad_norm";
    return guarded(fn, [&] { return norm_impl(fn, n, dtypes, numels, grads, counted, false, 0.0f, nullptr, workspace, norm, stream); });
}

int rtp_clip_grad_norm(int n, const int32_t* dtypes, const int64_t* numels, const void* const* grads,
                       const uint8_t* counted, float max_norm, void* const* out, void* workspace, float* norm,
                       rtp_stream stream)
{
    const char* fn = "rtp_clip_grad_norm";
    return guarded(fn, [&] { return norm_impl(fn, n, dtypes, numels, grads, counted, true, max_norm, out, workspace, norm, stream); });
}

}  // extern "C"
