// Global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum over counted tensors and their elements of g^2)
//   c    = min(1, max_norm / (norm + 1e-6)),   g' = c g
//
// HBM bound: every gradient is read for the norm, and read again and written for
// the product; what the second pass finds in L2 it need not read from HBM. Two
// kernels. The first leaves one float64 sum per block, and the last block to finish
// adds them up in block order (the sums of all blocks read by every block of the
// next kernel cost 6 us: one line of L2 for everyone). The second scales; it is a
// programmatic dependent of the first and has its first chunk in registers before
// that one has finished. Every block takes one run of chunks, forwards in the first
// kernel, backwards in the second, which so begins with what was read last. Runs and
// sums depend on the sizes and the device alone, so results are the same from run to
// run.
//
// Squares are added in float32 over a thread's part of one chunk (at most 64
// values, still in its registers) and across chunks in float64. A part whose
// float32 sum is outside [2^-60, 2^100] is added again in float64, so that the
// norm neither overflows nor underflows where it is itself a float32 number
// (below 2^-60 a lost square would matter, above 2^100 the next could overflow).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <vector>

#include "rtp_internal.h"

namespace rtp {

namespace {

constexpr int THREADS = 256, BLOCKS_PER_SM = 4;
constexpr int MAX_BLOCKS = 640;  // blocks, and partial sums, of one launch
// The scale kernel over more than this runs one block of 512 threads per SM: fewer
// streams of reads beside writes, and no streaming hints on them (805 MB: both passes
// 373 us, with hints 377; 101 MB, half of it in L2, 4 blocks of 256 with hints 51.7,
// without 54.2).
constexpr uint64_t WIDE_BYTES = 256u << 20;
constexpr int WIDE_THREADS = 512;

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
    uint16_t first[MAX_BLOCKS + 1];  // item of each block's first chunk, and of the end
    int32_t n;
    uint32_t chunks;
};
constexpr int SMALL = 64, LARGE = 512;  // tensors of one launch (3 KB or 18 KB of parameters)

__host__ __device__ __forceinline__ uint32_t run_begin(uint32_t chunks, int block, int blocks)
{
    return (uint32_t)((uint64_t)chunks * (uint32_t)block / (uint32_t)blocks);
}

// What the kernels share in the workspace. The counter is zero before the first call
// and zero again after every call.
struct Shared {
    unsigned finished;
    float norm;
    double partials[1];
};

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
    __syncthreads();  // a previous sum has been read
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) v += warp_sum[w];
    return v;
}

// Sum of the squares of V vectors (see the head of the file).
template <int V>
__device__ __forceinline__ double square_sum(const uint4 (&v)[V], bool bf16)
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) each(v[i], bf16, [&](float x) { s += x * x; });
    if (s >= 0x1p-60f && s <= 0x1p100f) return (double)s;
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) any |= v[i].x | v[i].y | v[i].z | v[i].w;
    double d = 0.0;
    if (any & (bf16 ? 0x7FFF7FFFu : 0x7FFFFFFFu)) {
#pragma unroll
        for (int i = 0; i < V; ++i) each(v[i], bf16, [&](float x) { d += (double)x * (double)x; });
    }
    return d;
}

// One chunk of the table: V vectors of 16 bytes for each of T threads. Tensors whose
// address is not a multiple of 16 have no vectors and go element by element, as do
// the elements after a tensor's last whole vector.
struct Chunk {
    const Item* it;
    bool bf16;
    int64_t e0;           // first element
    int left, nvec, per;  // elements, whole vectors, elements of a vector
};
template <int V, int T, int N>
__device__ __forceinline__ Chunk chunk_of(const Table<N>& t, int& item, uint32_t c, bool both)
{
    while (item + 1 < t.n && t.items[item + 1].chunk0 <= c) ++item;
    while (item > 0 && t.items[item].chunk0 > c) --item;
    Chunk k;
    k.it = &t.items[item];
    k.bf16 = k.it->dtype == RTP_BF16;
    k.per = k.bf16 ? 8 : 4;
    k.e0 = (int64_t)(c - k.it->chunk0) * (V * T * k.per);
    k.left = (int)min(k.it->numel - k.e0, (int64_t)(V * T * k.per));
    const uintptr_t at = (uintptr_t)k.it->src | (both ? (uintptr_t)k.it->dst : 0);
    k.nvec = (at & 15u) == 0 ? k.left / k.per : 0;
    return k;
}

// all: the partial sums of the launches so far, this one's at `begin`; the last
// launch's last block (last != 0) adds them all up.
template <int V, int N>
__global__ void __launch_bounds__(THREADS) grad_norm_kernel(const __grid_constant__ Table<N> t, Shared* sh, int begin,
                                                            int last, float* norm)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    double acc = 0.0;
    int item = t.first[blockIdx.x];
    const uint32_t c1 = run_begin(t.chunks, (int)blockIdx.x + 1, (int)gridDim.x);
    for (uint32_t c = run_begin(t.chunks, (int)blockIdx.x, (int)gridDim.x); c < c1; ++c) {
        const Chunk k = chunk_of<V, THREADS>(t, item, c, false);
        const uint4* p = static_cast<const uint4*>(k.it->src) + k.e0 / k.per;
        uint4 v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = i * THREADS + (int)threadIdx.x;
            v[i] = at < k.nvec ? __ldg(p + at) : make_uint4(0u, 0u, 0u, 0u);
        }
        for (int i = k.nvec * k.per + (int)threadIdx.x; i < k.left; i += THREADS) {
            const float x = k.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(k.it->src)[k.e0 + i])
                                   : static_cast<const float*>(k.it->src)[k.e0 + i];
            acc += (double)x * (double)x;
        }
        acc += square_sum<V>(v, k.bf16);
    }
    const double mine = block_sum(acc);
    __shared__ bool closing;
    if (threadIdx.x == 0) {
        sh->partials[begin + (int)blockIdx.x] = mine;
        closing = false;
        if (last) {
            __threadfence();
            closing = atomicAdd(&sh->finished, 1u) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!closing) return;
    // every block's sum is there (earlier launches' blocks are complete)
    __threadfence();
    double s = 0.0;
    for (int i = threadIdx.x; i < begin + (int)gridDim.x; i += THREADS) s += __ldcg(sh->partials + i);
    const float total = (float)sqrt(block_sum(s));
    if (threadIdx.x == 0) {
        sh->finished = 0u;
        sh->norm = total;
        *norm = total;
    }
}

__device__ __forceinline__ uint32_t scale2(uint32_t w, float c)
{
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(lo_f(w) * c)) |
           ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(hi_f(w) * c)) << 16);
}

__device__ __forceinline__ uint4 scaled(const uint4& v, bool bf16, float f)
{
    if (bf16) return make_uint4(scale2(v.x, f), scale2(v.y, f), scale2(v.z, f), scale2(v.w, f));
    return make_uint4(__float_as_uint(__uint_as_float(v.x) * f), __float_as_uint(__uint_as_float(v.y) * f),
                      __float_as_uint(__uint_as_float(v.z) * f), __float_as_uint(__uint_as_float(v.w) * f));
}

// (__ldg although the call may be in place: a chunk is read before its own block
// writes it, and by no other)
template <int V, int T, int N>
__global__ void __launch_bounds__(T) grad_scale_kernel(const __grid_constant__ Table<N> t, const Shared* sh, float max_norm,
                                                      int in_place)
{
    const uint32_t c0 = run_begin(t.chunks, (int)blockIdx.x, (int)gridDim.x);
    uint32_t c = run_begin(t.chunks, (int)blockIdx.x + 1, (int)gridDim.x);
    int item = t.first[blockIdx.x + 1];
    auto load = [&](const Chunk& k, uint4 (&v)[V]) {
        const uint4* p = static_cast<const uint4*>(k.it->src) + k.e0 / k.per;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = i * T + (int)threadIdx.x;
            if (at < k.nvec) v[i] = T == WIDE_THREADS ? __ldg(p + at) : __ldcs(p + at);
        }
    };
    uint4 v[V], next[V];
    Chunk k;
    if (c > c0) load(k = chunk_of<V, T>(t, item, c - 1, true), v);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float f = max_norm / (__ldcg(&sh->norm) + 1e-6f);
    if (f > 1.0f) f = 1.0f;  // a NaN stays one
    if (in_place && f == 1.0f) return;
    while (c > c0) {
        Chunk kn = k;
        if (c - 1 > c0) load(kn = chunk_of<V, T>(t, item, c - 2, true), next);
        uint4* q = static_cast<uint4*>(k.it->dst) + k.e0 / k.per;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = i * T + (int)threadIdx.x;
            if (at >= k.nvec) continue;
            if (T == WIDE_THREADS) q[at] = scaled(v[i], k.bf16, f);
            else __stcs(q + at, scaled(v[i], k.bf16, f));
        }
        for (int i = k.nvec * k.per + (int)threadIdx.x; i < k.left; i += T) {
            const int64_t e = k.e0 + i;
            if (k.bf16)
                static_cast<__nv_bfloat16*>(k.it->dst)[e] =
                    __float2bfloat16_rn(__bfloat162float(static_cast<const __nv_bfloat16*>(k.it->src)[e]) * f);
            else static_cast<float*>(k.it->dst)[e] = static_cast<const float*>(k.it->src)[e] * f;
        }
        --c;
        k = kn;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = next[i];
    }
}

// ---- host side --------------------------------------------------------------------

size_t esize(int dtype) { return dtype == RTP_F32 ? 4 : 2; }

// The launches of one pass over `items` (chunk0 not yet set), in chunks of
// chunk_bytes: call(table, blocks, index of launch, last one).
template <int N, class Call>
int each_launch(std::vector<Item>& items, uint64_t chunk_bytes, int blocks, Call&& call)
{
    static thread_local Table<N> t;
    size_t i = 0;
    for (int launch = 0; launch == 0 || i < items.size(); ++launch) {
        t.n = 0;
        uint64_t chunks = 0;
        for (; i < items.size() && t.n < N; ++i) {
            const uint64_t bytes = (uint64_t)items[i].numel * esize((int)items[i].dtype);
            const uint64_t add = (bytes + chunk_bytes - 1) / chunk_bytes;
            if (t.n > 0 && chunks + add > 0x7fffffffu) break;
            items[i].chunk0 = (uint32_t)chunks;
            t.items[t.n++] = items[i];
            chunks += add;
        }
        t.chunks = (uint32_t)chunks;
        const int grid = (int)std::max<uint64_t>(1, std::min<uint64_t>(chunks, (uint64_t)blocks));
        // item `it` holds the first chunk of the blocks b with run_begin(b) >= its chunk0,
        // that is b >= chunk0 * grid / chunks, up to the next item's
        for (int it = 0, b = 0; it < std::max(t.n, 1); ++it) {
            int end = grid + 1;
            if (it + 1 < t.n) {
                const uint64_t at = ((uint64_t)t.items[it + 1].chunk0 * (uint64_t)grid + t.chunks - 1) / t.chunks;
                end = (int)std::min<uint64_t>(at, (uint64_t)grid + 1);
            }
            for (; b < end; ++b) t.first[b] = (uint16_t)it;
        }
        int st = call(t, grid, launch, i >= items.size());
        if (st) return st;
    }
    return RTP_OK;
}

// The norm pass: V vectors a thread and chunk. Programmatic dependents of what ran
// before, which they wait for.
template <int V, int N>
int norm_pass(const char* fn, std::vector<Item>& counted, Shared* sh, float* norm, int blocks, cudaStream_t stream)
{
    int begin = 0;
    return each_launch<N>(counted, (uint64_t)V * THREADS * 16, blocks, [&](const Table<N>& t, int grid, int, bool last) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)grid);
        cfg.blockDim = dim3(THREADS);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cudaError_t e = cudaLaunchKernelEx(&cfg, grad_norm_kernel<V, N>, t, sh, begin, last ? 1 : 0, norm);
        begin += grid;
        return e == cudaSuccess ? RTP_OK : fail(RTP_ECUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
    });
}

// The scale pass. Its first launch is a programmatic dependent of the norm kernel,
// which announced it after its own wait: the gradients were written before either
// began. Later launches follow kernels that announce nothing.
template <int V, int T, int N>
int scale_pass(const char* fn, std::vector<Item>& all, const Shared* sh, float max_norm, bool in_place, int blocks,
               cudaStream_t stream)
{
    return each_launch<N>(all, (uint64_t)V * T * 16, blocks, [&](const Table<N>& t, int grid, int launch, bool) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)grid);
        cfg.blockDim = dim3(T);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = launch == 0 ? 1 : 0;
        cudaError_t e = cudaLaunchKernelEx(&cfg, grad_scale_kernel<V, T, N>, t, sh, max_norm, in_place ? 1 : 0);
        return e == cudaSuccess ? RTP_OK : fail(RTP_ECUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
    });
}

template <int N>
int run(const char* fn, std::vector<Item>& counted, std::vector<Item>& all, uint64_t bytes, Shared* sh, bool clip,
        float max_norm, bool in_place, float* norm, int sms, cudaStream_t s)
{
    // Chunks of 32 KB keep 8 loads in flight a thread; when there are too few of them
    // for every block, smaller ones spread the work over the SMs, and one block per SM
    // takes the norm: the blocks count themselves out on one word.
    const int blocks = std::min(sms * BLOCKS_PER_SM, MAX_BLOCKS);
    const bool fine = bytes / (uint64_t)blocks < 8u * THREADS * 16;
    int st = fine ? norm_pass<2, N>(fn, counted, sh, norm, std::min(sms, MAX_BLOCKS), s)
                  : norm_pass<8, N>(fn, counted, sh, norm, blocks, s);
    if (st || !clip || all.empty()) return st;
    if (bytes >= WIDE_BYTES) return scale_pass<8, WIDE_THREADS, N>(fn, all, sh, max_norm, in_place, std::min(sms, MAX_BLOCKS), s);
    if (fine) return scale_pass<1, THREADS, N>(fn, all, sh, max_norm, in_place, blocks, s);
    return scale_pass<4, THREADS, N>(fn, all, sh, max_norm, in_place, blocks, s);
}

// One launch for each LARGE tensors (and for each 2^31 chunks, 8 TB: never).
int64_t workspace_bytes(int n) { return 16 + (int64_t)(n / LARGE + 1) * MAX_BLOCKS * 8; }

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
    in.reserve((size_t)n);
    all.reserve((size_t)n);
    ranges.reserve((size_t)n * 2);
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
    int sms = 0;
    if (device_sms(&sms)) return fail(RTP_ECUDA, "%s: no CUDA device", fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Shared* sh = static_cast<Shared*>(workspace);
    if (all.size() <= SMALL) return run<SMALL>(fn, in, all, bytes, sh, clip, max_norm, in_place, norm, sms, s);
    return run<LARGE>(fn, in, all, bytes, sh, clip, max_norm, in_place, norm, sms, s);
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
