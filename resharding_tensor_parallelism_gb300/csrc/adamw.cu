// AdamW step over many tensors at once (rank pieces of weights), moments in float32 or
// in 8 bits:
//
//   g' = c g, c = min(1, max_norm / (norm + 1e-6))      (clipping by a norm on the device)
//   m = b1 m + (1 - b1) g'    v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// HBM bound: every value is read and written once (bf16 weights with a float32 copy and
// bf16 gradients: 28 bytes an element with float32 moments, 16 with 8-bit ones). The
// step count, its powers and the corrections are on the device, so that a captured step
// counts on with every replay: the last block to finish a step advances them.
//
// A warp takes rows of 128 elements, 4 to a lane: 16-byte accesses of float32, 8 of bf16,
// 4 of 8-bit moments, all of them whole lines. A row is a block of the 8-bit format, so
// a block's largest value is one warp reduction.
//
// 8-bit moments (128 elements share a power of two; an exponent byte E of the block's
// largest absolute value, at least 27, as in a float32; 255: everything is NaN):
//   m  sign, 4 bits of exponent, 3 of mantissa: value (1 + M/8) 2^(e-7), e = 0: M/8 2^-6,
//      times 2^(E-134): the largest has the exponent 7, 2^-17.8 of it is the least
//   v  5 bits of exponent, 3 of mantissa: (1 + M/8) 2^(e-15), e = 0: M/8 2^-14, times
//      2^(E-142): down to 2^-33 of the largest; what is not zero never becomes zero, or
//      the next step would divide by eps
// Values are rounded up or down at random, with the probabilities that keep the mean
// (rounding to nearest would leave v as it is: a step changes it by 1 - b2, less than
// half a spacing). A bf16 weight without a float32 copy is rounded the same way, or small
// steps would be lost. The bits are a hash of seed, tensor, step and element: a step is
// reproducible bit for bit. The update itself uses m and v before they are rounded.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <vector>

#include "rtp_internal.h"

namespace rtp {

namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int ROW = RTP_ADAMW_BLOCK;  // elements of a warp's row, and of a block of 8-bit moments
static_assert(ROW == 128, "4 elements a lane");
constexpr int LEAST_EXPONENT = 27;

struct Item {
    void* param;
    const void* grad;
    float* master;
    void* m;
    void* v;
    uchar2* scales;
    int64_t numel;
    uint32_t chunk0;  // first chunk
    float decay;
    uint32_t id;
    uint8_t param_bf16, grad_bf16, vectors, unused;
};
template <int N>
struct Table {
    Item items[N];
    int32_t n;
    uint32_t chunks;
};
constexpr int SMALL = 32, LARGE = 256;  // tensors of one launch (2.3 KB or 18 KB of parameters)

// On the device; rtp_adamw_clock writes it, a step advances it.
struct Clock {
    long long step;         // steps done
    double power1, power2;  // b1^(step + 1), b2^(step + 1)
    double beta1, beta2;
    float correct1, correct2;          // 1 / (1 - power)
    float keep1, keep2, rest1, rest2;  // b1, b2, 1 - b1, 1 - b2
    unsigned finished;
};
static_assert(sizeof(Clock) <= RTP_ADAMW_CLOCK_BYTES, "");

struct Step {
    Clock* clock;
    const float* lr_at;  // or NULL
    const float* norm;   // or NULL
    float lr, max_norm, eps;
    uint32_t seed;
    int32_t last;  // launch of the step
};

// A 32-bit hash: the output function of PCG-RXS-M-XS 32/32 on one step of its state
// (M. O'Neill, "PCG: A Family of Simple Fast Space-Efficient Statistically Good
// Algorithms for Random Number Generation", 2014).
__device__ __forceinline__ uint32_t pcg(uint32_t x)
{
    x = x * 747796405u + 2891336453u;
    const uint32_t w = ((x >> ((x >> 28) + 4u)) ^ x) * 277803737u;
    return (w >> 22) ^ w;
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float power_of_two(int biased) { return __uint_as_float((uint32_t)biased << 23); }

// 2^(E - base) of a block's exponent byte, or NaN.
__device__ __forceinline__ float block_scale(int e, int base)
{
    return e == 255 ? __int_as_float(0x7FC00000) : power_of_two(max(e, LEAST_EXPONENT) - base + 127);
}
__device__ __forceinline__ float decode_m(uint32_t code, float scale)
{
    const float z = __uint_as_float((code & 127u) << 20) * 0x1p120f * scale;
    return __uint_as_float(__float_as_uint(z) | (code & 128u) << 24);
}
__device__ __forceinline__ float decode_v(uint32_t code, float scale) { return __uint_as_float(code << 20) * 0x1p112f * scale; }

// z >= 0 in a format of 3 mantissa bits and this bias, its lost 20 bits rounded up when
// they and `r` (20 bits) carry. Below the smallest normal value that value is added, so
// that the codes' spacing there is the one of its binade.
template <int BIAS>
__device__ __forceinline__ uint32_t encode(float z, uint32_t r)
{
    constexpr float LEAST = BIAS == 7 ? 0x1p-6f : 0x1p-14f;
    const bool low = z < LEAST;
    const uint32_t bits = __float_as_uint(low ? z + LEAST : z);
    return ((bits + r) >> 20) - (uint32_t)((127 - BIAS) << 3) - (low ? 8u : 0u);
}

// 4 elements of type f32 or bf16 as they are in memory, bf16 in two words.
struct Raw {
    uint4 w;
};
__device__ __forceinline__ Raw load4(const void* p, bool bf16, int64_t at, int n, bool vectors)
{
    Raw r = {make_uint4(0u, 0u, 0u, 0u)};
    if (vectors && n >= 4) {
        if (bf16) {
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(static_cast<const char*>(p) + 2 * at));
            r.w.x = v.x, r.w.y = v.y;
        } else {
            r.w = __ldcs(reinterpret_cast<const uint4*>(static_cast<const char*>(p) + 4 * at));
        }
    } else if (bf16) {
        const unsigned short* q = static_cast<const unsigned short*>(p) + at;
        if (n > 0) r.w.x = q[0];
        if (n > 1) r.w.x |= (uint32_t)q[1] << 16;
        if (n > 2) r.w.y = q[2];
        if (n > 3) r.w.y |= (uint32_t)q[3] << 16;
    } else {
        const uint32_t* q = static_cast<const uint32_t*>(p) + at;
        if (n > 0) r.w.x = q[0];
        if (n > 1) r.w.y = q[1];
        if (n > 2) r.w.z = q[2];
        if (n > 3) r.w.w = q[3];
    }
    return r;
}
__device__ __forceinline__ void floats(const Raw& r, bool bf16, float (&x)[4])
{
    x[0] = bf16 ? lo_f(r.w.x) : __uint_as_float(r.w.x);
    x[1] = bf16 ? hi_f(r.w.x) : __uint_as_float(r.w.y);
    x[2] = bf16 ? lo_f(r.w.y) : __uint_as_float(r.w.z);
    x[3] = bf16 ? hi_f(r.w.y) : __uint_as_float(r.w.w);
}
__device__ __forceinline__ void store_f32(void* p, int64_t at, int n, bool vectors, const float (&x)[4])
{
    float* q = static_cast<float*>(p) + at;
    if (vectors && n >= 4) {
        __stcs(reinterpret_cast<float4*>(q), make_float4(x[0], x[1], x[2], x[3]));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < n) q[j] = x[j];
    }
}
__device__ __forceinline__ void store_16(void* p, int64_t at, int n, bool vectors, const uint32_t (&x)[4])
{
    unsigned short* q = static_cast<unsigned short*>(p) + at;
    if (vectors && n >= 4) {
        __stcs(reinterpret_cast<uint2*>(q), make_uint2(x[0] | x[1] << 16, x[2] | x[3] << 16));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < n) q[j] = (unsigned short)x[j];
    }
}
__device__ __forceinline__ uint32_t load_codes(const void* p, int64_t at, int n, bool vectors)
{
    const uint8_t* q = static_cast<const uint8_t*>(p) + at;
    if (vectors && n >= 4) return __ldcs(reinterpret_cast<const unsigned int*>(q));
    uint32_t w = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n) w |= (uint32_t)q[j] << 8 * j;
    return w;
}
__device__ __forceinline__ void store_codes(void* p, int64_t at, int n, bool vectors, uint32_t w)
{
    uint8_t* q = static_cast<uint8_t*>(p) + at;
    if (vectors && n >= 4) {
        __stcs(reinterpret_cast<unsigned int*>(q), w);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < n) q[j] = (uint8_t)(w >> 8 * j);
    }
}

__device__ __forceinline__ uint32_t round_bf16(float x) { return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x)); }
// Up when the lost 16 bits and r (16 bits) carry; NaN and infinity stay.
__device__ __forceinline__ uint32_t round_bf16_at_random(float x, uint32_t r)
{
    return fabsf(x) < __int_as_float(0x7F800000) ? (__float_as_uint(x) + r) >> 16 : round_bf16(x);
}
__device__ __forceinline__ float sqrt_fast(float x)
{
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Rows of a thread in flight: ROWS; a chunk is what a block takes at once.
template <int ROWS>
constexpr int CHUNK = ROWS * WARPS * ROW;

template <bool BITS8, int ROWS, int N>
__global__ void __launch_bounds__(THREADS, 2) adamw_kernel(const __grid_constant__ Table<N> t, const __grid_constant__ Step s)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float beta1 = s.clock->keep1, beta2 = s.clock->keep2, rest1 = s.clock->rest1, rest2 = s.clock->rest2;
    const float correct2 = s.clock->correct2, lr = s.lr_at ? __ldcg(s.lr_at) : s.lr, rate = lr * s.clock->correct1;
    const uint32_t step = (uint32_t)(s.clock->step + 1);
    float clip = 1.0f;
    if (s.norm) {
        clip = s.max_norm / (__ldcg(s.norm) + 1e-6f);
        if (clip > 1.0f) clip = 1.0f;  // a NaN stays one
    }
    int item = 0;
    for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        for (int half = N / 2; half > 0; half /= 2)
            if (item + half < t.n && t.items[item + half].chunk0 <= c) item += half;
        const Item& it = t.items[item];
        const bool pb = it.param_bf16, gb = it.grad_bf16, vec = it.vectors;
        const int64_t e0 = (int64_t)(c - it.chunk0) * CHUNK<ROWS> + warp * ROW;  // row i: WARPS * ROW further on
        Raw p[ROWS], g[ROWS], m[ROWS], v[ROWS];
        uchar2 scales[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int64_t row = e0 + i * (WARPS * ROW), at = row + 4 * lane;
            const int n = (int)min((int64_t)4, it.numel - at);
            p[i] = it.master ? load4(it.master, false, at, n, vec) : load4(it.param, pb, at, n, vec);
            g[i] = load4(it.grad, gb, at, n, vec);
            if constexpr (BITS8) {
                m[i].w.x = load_codes(it.m, at, n, vec);
                v[i].w.x = load_codes(it.v, at, n, vec);
                scales[i] = row < it.numel ? __ldcs(it.scales + row / ROW) : make_uchar2(0, 0);
            } else {
                m[i] = load4(it.m, false, at, n, vec);
                v[i] = load4(it.v, false, at, n, vec);
            }
        }
        const uint32_t key = pcg(pcg(pcg(s.seed) + it.id) + step);
        const float keep = 1.0f - lr * it.decay;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int64_t row = e0 + i * (WARPS * ROW), at = row + 4 * lane;
            if (row >= it.numel) break;  // the warp's
            const int n = (int)min((int64_t)4, it.numel - at);
            float x[4], dx[4], m1[4], v1[4];
            floats(p[i], pb && !it.master, x);
            floats(g[i], gb, dx);
            if constexpr (BITS8) {
                const float ms = block_scale(scales[i].x, 134), vs = block_scale(scales[i].y, 142);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    m1[j] = decode_m(m[i].w.x >> 8 * j & 255u, ms);
                    v1[j] = decode_v(v[i].w.x >> 8 * j & 255u, vs);
                }
            } else {
                floats(m[i], false, m1);
                floats(v[i], false, v1);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float d = dx[j] * clip;
                m1[j] = fmaf(beta1, m1[j], rest1 * d);
                v1[j] = fmaf(beta2, v1[j], rest2 * d * d);
                x[j] = fmaf(x[j], keep, -rate * __fdividef(m1[j], sqrt_fast(v1[j] * correct2) + s.eps));
            }
            uint32_t noise[4];
            if (BITS8 || (pb && !it.master)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) noise[j] = pcg((uint32_t)at + (uint32_t)j + key);
            }
            if (it.master) store_f32(it.master, at, n, vec, x);
            if (!pb) {
                store_f32(it.param, at, n, vec, x);
            } else {
                uint32_t b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = it.master ? round_bf16(x[j]) : round_bf16_at_random(x[j], pcg(noise[j]) & 0xFFFFu);
                store_16(it.param, at, n, vec, b);
            }
            if constexpr (BITS8) {
                uint32_t mt = 0u, vt = 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // elements behind the end count as 0
                    mt = max(mt, j < n ? __float_as_uint(fabsf(m1[j])) : 0u);
                    vt = max(vt, j < n ? __float_as_uint(fabsf(v1[j])) : 0u);
                }
                const int me = max((int)(__reduce_max_sync(0xffffffffu, mt) >> 23), LEAST_EXPONENT);
                const int ve = max((int)(__reduce_max_sync(0xffffffffu, vt) >> 23), LEAST_EXPONENT);
                const float ms = power_of_two(261 - me), vs = power_of_two(269 - ve);  // 2^(134 - E), 2^(142 - E)
                uint32_t mc = 0u, vc = 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a = encode<7>(fabsf(m1[j]) * ms, (noise[j] & 0xFFFFu) << 4 | 8u) & 127u;
                    const uint32_t b = max(encode<15>(v1[j] * vs, noise[j] >> 16 << 4 | 8u) & 255u, v1[j] > 0.0f ? 1u : 0u);
                    mc |= (a | (__float_as_uint(m1[j]) >> 31 << 7)) << 8 * j;
                    vc |= b << 8 * j;
                }
                store_codes(it.m, at, n, vec, mc);
                store_codes(it.v, at, n, vec, vc);
                if (lane == 0) it.scales[row / ROW] = make_uchar2((unsigned char)me, (unsigned char)ve);
            } else {
                store_f32(it.m, at, n, vec, m1);
                store_f32(it.v, at, n, vec, v1);
            }
        }
    }
    if (!s.last) return;
    __syncthreads();  // every thread has read the clock
    if (threadIdx.x == 0 && atomicAdd(&s.clock->finished, 1u) == gridDim.x - 1) {
        Clock& k = *s.clock;
        k.finished = 0u;
        k.step += 1;
        k.power1 *= k.beta1;
        k.power2 *= k.beta2;
        k.correct1 = (float)(1.0 / (1.0 - k.power1));
        k.correct2 = (float)(1.0 / (1.0 - k.power2));
    }
}

__global__ void adamw_clock_kernel(Clock* k, long long step, double beta1, double beta2)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    k->step = step;
    k->beta1 = beta1;
    k->beta2 = beta2;
    k->power1 = pow(beta1, (double)(step + 1));
    k->power2 = pow(beta2, (double)(step + 1));
    k->correct1 = (float)(1.0 / (1.0 - k->power1));
    k->correct2 = (float)(1.0 / (1.0 - k->power2));
    k->keep1 = (float)beta1;
    k->keep2 = (float)beta2;
    k->rest1 = (float)(1.0 - beta1);
    k->rest2 = (float)(1.0 - beta2);
    k->finished = 0u;
}

// Values of 8-bit moments: 16 elements a thread, 8 threads a block of the format.
template <bool F32>
__global__ void __launch_bounds__(THREADS) adamw_values_kernel(const uint4* m8, const uint4* v8, const uchar2* scales, void* m,
                                                               void* v, int64_t units)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t stride = (int64_t)gridDim.x * THREADS;
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < units; i += stride) {
        const uchar2 sc = scales[i / (ROW / 16)];
        const float ms = block_scale(sc.x, 134), vs = block_scale(sc.y, 142);
        const uint4 a = __ldcs(m8 + i), b = __ldcs(v8 + i);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
        float x[16], y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            x[j] = decode_m(aw[j / 4] >> 8 * (j % 4) & 255u, ms);
            y[j] = decode_v(bw[j / 4] >> 8 * (j % 4) & 255u, vs);
        }
        if constexpr (F32) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                static_cast<float4*>(m)[4 * i + q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
                static_cast<float4*>(v)[4 * i + q] = make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
            }
        } else {
            uint32_t p[8], q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p[j] = round_bf16(x[2 * j]) | round_bf16(x[2 * j + 1]) << 16;
                q[j] = round_bf16(y[2 * j]) | round_bf16(y[2 * j + 1]) << 16;
            }
            static_cast<uint4*>(m)[2 * i] = make_uint4(p[0], p[1], p[2], p[3]);
            static_cast<uint4*>(m)[2 * i + 1] = make_uint4(p[4], p[5], p[6], p[7]);
            static_cast<uint4*>(v)[2 * i] = make_uint4(q[0], q[1], q[2], q[3]);
            static_cast<uint4*>(v)[2 * i + 1] = make_uint4(q[4], q[5], q[6], q[7]);
        }
    }
}

// ---- host side --------------------------------------------------------------------

template <class... A, class... B>
int launch(const char* fn, void (*kernel)(A...), unsigned grid, int threads, cudaStream_t stream, B... args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? RTP_OK : fail(RTP_ECUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
}

// Table by table, in chunks of ROWS rows a warp. The step's clock moves on with the last
// one, which runs (on one block) even when there is nothing to update.
template <bool BITS8, int ROWS, int N>
int run(const char* fn, std::vector<Item>& items, Step s, int blocks, cudaStream_t stream)
{
    static thread_local Table<N> t;
    size_t i = 0;
    do {
        t.n = 0;
        uint64_t chunks = 0;
        for (; i < items.size() && t.n < N; ++i) {
            const uint64_t add = ((uint64_t)items[i].numel + CHUNK<ROWS> - 1) / CHUNK<ROWS>;
            if (t.n > 0 && chunks + add > 0x7fffffffu) break;
            items[i].chunk0 = (uint32_t)chunks;
            t.items[t.n++] = items[i];
            chunks += add;
        }
        t.chunks = (uint32_t)chunks;
        s.last = i >= items.size();
        const unsigned grid = (unsigned)std::max<uint64_t>(1, std::min<uint64_t>(chunks, (uint64_t)blocks));
        const int st = launch(fn, adamw_kernel<BITS8, ROWS, N>, grid, THREADS, stream, t, s);
        if (st) return st;
    } while (i < items.size());
    return RTP_OK;
}

int step_impl(const char* fn, int n, const rtp_adamw_tensor* tensors, int bits, float lr, const float* lr_at, float eps,
              const float* norm, float max_norm, uint32_t seed, void* clock, cudaStream_t stream)
{
    if (n < 0 || (n > 0 && !tensors)) return fail(RTP_EINVAL, "%s: n = %d, or NULL tensors", fn, n);
    if (bits != 32 && bits != 8) return fail(RTP_EINVAL, "%s: moments of %d bits (32 or 8)", fn, bits);
    if (!clock || ((uintptr_t)clock & 15u)) return fail(RTP_EINVAL, "%s: the clock must be there and 16-byte aligned", fn);
    if (((uintptr_t)lr_at | (uintptr_t)norm) & 3u) return fail(RTP_EINVAL, "%s: lr or norm is not aligned to its elements", fn);
    if (!lr_at && !(lr >= 0.0f)) return fail(RTP_EINVAL, "%s: lr %g is not a number >= 0", fn, (double)lr);
    if (!(eps >= 0.0f)) return fail(RTP_EINVAL, "%s: eps %g is not a number >= 0", fn, (double)eps);
    if (norm && !(max_norm >= 0.0f)) return fail(RTP_EINVAL, "%s: max_norm %g is not a number >= 0", fn, (double)max_norm);
    std::vector<Item> items;
    items.reserve((size_t)n);
    std::vector<std::pair<uintptr_t, uintptr_t>> written;
    written.reserve((size_t)n * 2);
    uint64_t elements = 0;
    for (int i = 0; i < n; ++i) {
        const rtp_adamw_tensor& w = tensors[i];
        if ((w.param_dtype != RTP_F32 && w.param_dtype != RTP_BF16) || (w.grad_dtype != RTP_F32 && w.grad_dtype != RTP_BF16))
            return fail(RTP_EINVAL, "%s: tensor %d is of an unknown type", fn, i);
        if (w.numel < 0 || w.numel >= (int64_t)1 << 42) return fail(RTP_ESHAPE, "%s: tensor %d has %lld elements", fn, i, (long long)w.numel);
        if (!(w.weight_decay >= 0.0f)) return fail(RTP_EINVAL, "%s: weight decay %g of tensor %d is not a number >= 0", fn, (double)w.weight_decay, i);
        if (w.numel == 0) continue;
        const bool pb = w.param_dtype == RTP_BF16, gb = w.grad_dtype == RTP_BF16;
        if (!w.param || !w.grad || !w.exp_avg || !w.exp_avg_sq || (bits == 8 && !w.scales))
            return fail(RTP_EINVAL, "%s: NULL buffer of tensor %d", fn, i);
        if (w.master && !pb) return fail(RTP_EINVAL, "%s: tensor %d is float32 and has a float32 copy", fn, i);
        const uintptr_t f32s = (uintptr_t)w.master | (pb ? 0 : (uintptr_t)w.param) | (gb ? 0 : (uintptr_t)w.grad) |
                               (bits == 8 ? 0 : (uintptr_t)w.exp_avg | (uintptr_t)w.exp_avg_sq);
        const uintptr_t b16s = (pb ? (uintptr_t)w.param : 0) | (gb ? (uintptr_t)w.grad : 0);
        const uintptr_t b8s = bits == 8 ? (uintptr_t)w.exp_avg | (uintptr_t)w.exp_avg_sq : 0;
        if ((f32s & 3u) || (b16s & 1u) || (bits == 8 && ((uintptr_t)w.scales & 1u)))
            return fail(RTP_EINVAL, "%s: a buffer of tensor %d is not aligned to its elements", fn, i);
        Item it = {w.param, w.grad, w.master, w.exp_avg, w.exp_avg_sq, reinterpret_cast<uchar2*>(w.scales), w.numel, 0u,
                   w.weight_decay, (uint32_t)i, pb, gb, (uint8_t)(!(f32s & 15u) && !(b16s & 7u) && !(b8s & 3u)), 0};
        items.push_back(it);
        elements += (uint64_t)w.numel;
        const uintptr_t p = (uintptr_t)w.param;
        written.emplace_back(p, p + (uint64_t)w.numel * (pb ? 2 : 4));
        if (w.master) written.emplace_back((uintptr_t)w.master, (uintptr_t)w.master + (uint64_t)w.numel * 4);
    }
    std::sort(written.begin(), written.end());
    for (size_t i = 1; i < written.size(); ++i)
        if (written[i - 1].second > written[i].first) return fail(RTP_EINVAL, "%s: weights or their copies share bytes", fn);
    int sms = 0;
    if (device_sms(&sms)) return fail(RTP_ECUDA, "%s: no CUDA device", fn);
    const Step s = {static_cast<Clock*>(clock), lr_at, norm, lr, max_norm, eps, seed, 0};
    const int blocks = sms * 2;
    const bool fine = elements < (uint64_t)blocks * CHUNK<4>;  // one row a warp spreads them over the GPU
    auto go = [&](auto wide) {
        constexpr bool B8 = decltype(wide)::value;
        if (items.size() <= SMALL)
            return fine ? run<B8, 1, SMALL>(fn, items, s, blocks, stream) : run<B8, 4, SMALL>(fn, items, s, blocks, stream);
        return fine ? run<B8, 1, LARGE>(fn, items, s, blocks, stream) : run<B8, 4, LARGE>(fn, items, s, blocks, stream);
    };
    return bits == 8 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace

}  // namespace rtp

using namespace rtp;

extern "C" {

int rtp_adamw_clock(void* clock, int64_t step, double beta1, double beta2, rtp_stream stream)
{
    const char* fn = "rtp_adamw_clock";
    if (!clock || ((uintptr_t)clock & 15u)) return fail(RTP_EINVAL, "%s: the clock must be there and 16-byte aligned", fn);
    if (step < 0) return fail(RTP_EINVAL, "%s: step %lld", fn, (long long)step);
    if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0))
        return fail(RTP_EINVAL, "%s: betas %g and %g outside [0, 1)", fn, beta1, beta2);
    return launch(fn, adamw_clock_kernel, 1, 1, static_cast<cudaStream_t>(stream), static_cast<Clock*>(clock), (long long)step,
                  beta1, beta2);
}

int rtp_adamw_step(int n, const rtp_adamw_tensor* tensors, int bits, float lr, const float* lr_at, float eps, const float* norm,
                   float max_norm, uint32_t seed, void* clock, rtp_stream stream)
{
    const char* fn = "rtp_adamw_step";
    return guarded(fn, [&] {
        return step_impl(fn, n, tensors, bits, lr, lr_at, eps, norm, max_norm, seed, clock, static_cast<cudaStream_t>(stream));
    });
}

int rtp_adamw_values(int64_t blocks, const uint8_t* exp_avg, const uint8_t* exp_avg_sq, const uint8_t* scales, rtp_dtype dtype,
                     void* m, void* v, rtp_stream stream)
{
    const char* fn = "rtp_adamw_values";
    if (blocks < 0 || blocks >= (int64_t)1 << 42) return fail(RTP_ESHAPE, "%s: %lld blocks", fn, (long long)blocks);
    if (dtype != RTP_F32 && dtype != RTP_BF16) return fail(RTP_EINVAL, "%s: unknown type %d", fn, dtype);
    if (blocks == 0) return RTP_OK;
    if (!exp_avg || !exp_avg_sq || !scales || !m || !v) return fail(RTP_EINVAL, "%s: NULL argument", fn);
    if ((((uintptr_t)exp_avg | (uintptr_t)exp_avg_sq | (uintptr_t)m | (uintptr_t)v) & 15u) || ((uintptr_t)scales & 1u))
        return fail(RTP_EINVAL, "%s: a buffer is not 16-byte aligned", fn);
    int sms = 0;
    if (device_sms(&sms)) return fail(RTP_ECUDA, "%s: no CUDA device", fn);
    const int64_t units = blocks * (ROW / 16);
    const unsigned grid = (unsigned)std::min<int64_t>((units + THREADS - 1) / THREADS, (int64_t)sms * 8);
    return launch(fn, dtype == RTP_F32 ? adamw_values_kernel<true> : adamw_values_kernel<false>, grid, THREADS,
                  static_cast<cudaStream_t>(stream), reinterpret_cast<const uint4*>(exp_avg),
                  reinterpret_cast<const uint4*>(exp_avg_sq), reinterpret_cast<const uchar2*>(scales), m, v, units);
}

}  // extern "C"
