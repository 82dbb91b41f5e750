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
// Measured on 201 M elements in 25 tensors of that kind: float32 moments 858 us (97 % of
// the copy rate), 8-bit ones 620 (bound by their arithmetic); 1.6 M float32 elements 9.4 us.
//
// A warp takes rows of 128 elements, 4 to a lane: 16-byte accesses of float32, 8 of bf16,
// 4 of 8-bit moments, all of them whole lines. A row is a block of the 8-bit format, so
// a block's largest value is one warp reduction.
//
// 8-bit moments (128 elements share a power of two; an exponent byte E of the block's
// largest absolute value, at least 27, as in a float32; 255: everything is NaN):
//   m  sign, 4 bits of exponent, 3 of mantissa: value (1 + M/8) 2^(e-7), e = 0: M/8 2^-6,
//      times 2^(E-134): the largest has the exponent 7, the least is 2^-16 to 2^-17 of it
//   v  5 bits of exponent, 3 of mantissa: (1 + M/8) 2^(e-15), e = 0: M/8 2^-14, times
//      2^(E-142): the least is 2^-32 to 2^-33 of the largest; what is not zero never becomes zero, or
//      the next step would divide by eps
// Values are rounded up or down at random, with the probabilities that keep the mean
// (rounding to nearest would leave v as it is: a step changes it by 1 - b2, less than
// half a spacing). A bf16 weight without a float32 copy is rounded the same way, or small
// steps would be lost. The bits are a hash of seed, tensor, step and element: a step is
// reproducible bit for bit (replicas of a tensor are given the same number instead of their
// places, and stay alike). The update itself uses m and v before they are rounded. They are
// formed by single float32 operations (no fused ones), so that any float32 program gets
// the same codes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <vector>

#include "launch.cuh"
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
    uint32_t id;  // of its random bits
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
__device__ __forceinline__ float sqrt_ftz(float x)
{
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_ftz(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// What a step has read from the device, and its launch's arguments.
struct Rates {
    float beta1, beta2, rest1, rest2, correct2, lr, rate, clip, eps;
    uint32_t seed, step;
};

// A weight behind its moments. The second form goes with the blocks of 8-bit moments whose exponents are
// no larger than these: it takes fewer instructions, and the denominator is formed times 2^32, so that no v but 0
// counts as zero. Which of them a weight takes depends on its values alone, not on its place in memory: replicas
// that are given the same stay the same.
constexpr int MOST_M = 140, MOST_V = 156;
__device__ __forceinline__ float updated(float x, float keep, float m, float v, const Rates& s)
{
    return fmaf(x, keep, -s.rate * __fdividef(m, sqrt_fast(v * s.correct2) + s.eps));
}
__device__ __forceinline__ float updated_scaled(float x, float keep, float m, float v, const Rates& s)
{
    return fmaf(x, keep, s.rate * -0x1p32f * m * rcp_ftz(sqrt_ftz(v * (s.correct2 * 0x1p64f)) + s.eps * 0x1p32f));
}

// One row of any types, alignment and length.
template <bool BITS8>
__device__ __noinline__ void any_row(const Item& it, int64_t row, const Rates& s)
{
    const int lane = threadIdx.x & 31;
    const bool pb = it.param_bf16, gb = it.grad_bf16, vec = it.vectors;
    const int64_t at = row + 4 * lane;
    const int n = (int)min((int64_t)4, it.numel - at);
    const uint32_t key = pcg(pcg(pcg(s.seed) + it.id) + s.step);
    const float keep = 1.0f - s.lr * it.decay;
    float x[4], dx[4], m[4], v[4];
    bool scaled = BITS8;
    floats(it.master ? load4(it.master, false, at, n, vec) : load4(it.param, pb, at, n, vec), pb && !it.master, x);
    floats(load4(it.grad, gb, at, n, vec), gb, dx);
    if constexpr (BITS8) {
        const uint32_t mw = load_codes(it.m, at, n, vec), vw = load_codes(it.v, at, n, vec);
        const uchar2 scales = __ldcs(it.scales + row / ROW);
        const float ms = block_scale(scales.x, 134), vs = block_scale(scales.y, 142);
        scaled = scales.x <= MOST_M && scales.y <= MOST_V;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m[j] = decode_m(mw >> 8 * j & 255u, ms);
            v[j] = decode_v(vw >> 8 * j & 255u, vs);
        }
        __syncwarp();  // the block's exponents have been read
    } else {
        floats(load4(it.m, false, at, n, vec), false, m);
        floats(load4(it.v, false, at, n, vec), false, v);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float d = dx[j] * s.clip;
        m[j] = BITS8 ? __fadd_rn(__fmul_rn(s.beta1, m[j]), __fmul_rn(s.rest1, d)) : fmaf(s.beta1, m[j], s.rest1 * d);
        v[j] = BITS8 ? __fadd_rn(__fmul_rn(s.beta2, v[j]), __fmul_rn(__fmul_rn(s.rest2, d), d)) : fmaf(s.beta2, v[j], s.rest2 * d * d);
    }
    int me = 0, ve = 0;  // exponents of the block's largest
    if constexpr (BITS8) {
        uint32_t mt = 0u, vt = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // elements behind the end count as 0
            mt = max(mt, j < n ? __float_as_uint(fabsf(m[j])) : 0u);
            vt = max(vt, j < n ? __float_as_uint(fabsf(v[j])) : 0u);
        }
        me = max((int)(__reduce_max_sync(0xffffffffu, mt) >> 23), LEAST_EXPONENT);
        ve = max((int)(__reduce_max_sync(0xffffffffu, vt) >> 23), LEAST_EXPONENT);
        scaled = scaled && me <= MOST_M && ve <= MOST_V;
    }
    uint32_t noise[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = scaled ? updated_scaled(x[j], keep, m[j], v[j], s) : updated(x[j], keep, m[j], v[j], s);
        noise[j] = pcg((uint32_t)at + (uint32_t)j + key);
        b[j] = it.master ? round_bf16(x[j]) : round_bf16_at_random(x[j], pcg(noise[j]) & 0xFFFFu);
    }
    if (it.master) store_f32(it.master, at, n, vec, x);
    if (pb) store_16(it.param, at, n, vec, b);
    else store_f32(it.param, at, n, vec, x);
    if constexpr (BITS8) {
        const float ms = power_of_two(261 - me), vs = power_of_two(269 - ve);  // 2^(134 - E), 2^(142 - E)
        uint32_t mc = 0u, vc = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a = encode<7>(fabsf(m[j]) * ms, (noise[j] & 0xFFFFu) << 4 | 8u) & 127u;
            const uint32_t c = max(encode<15>(v[j] * vs, noise[j] >> 16 << 4 | 8u) & 255u, v[j] > 0.0f ? 1u : 0u);
            mc |= (a | (__float_as_uint(m[j]) >> 31 << 7)) << 8 * j;
            vc |= c << 8 * j;
        }
        store_codes(it.m, at, n, vec, mc);
        store_codes(it.v, at, n, vec, vc);
        if (lane == 0) it.scales[row / ROW] = make_uchar2((unsigned char)me, (unsigned char)ve);
    } else {
        store_f32(it.m, at, n, vec, m);
        store_f32(it.v, at, n, vec, v);
    }
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Whole, aligned rows of 8-bit moments: the row's update in as few instructions as the
// format allows (in the form of any_row, 200 an element, the arithmetic took 2.3 times as
// long as the memory). A code shifted to the bits that a float32's exponent and mantissa
// end in, subnormal ones too, is the value it stands for times a power of two, which goes
// into beta's factor; a value times a power of two has its code in those bits, with the
// lost part below. Both hold for block exponents that such powers of two fit; other
// rows (and NaN) return false with nothing written.
template <bool PB, bool MASTER, bool GB>
__device__ __forceinline__ bool row_of_8_bits(const Item& it, int64_t at, const Raw& p, const Raw& g, uint32_t mw, uint32_t vw,
                                              uchar2 scales, const Rates& s, float keep, uint32_t key)
{
    const int em = max((int)scales.x, LEAST_EXPONENT), ev = max((int)scales.y, LEAST_EXPONENT);
    if (em > MOST_M || ev > MOST_V) return false;
    const float fm = s.beta1 * power_of_two(em - 14 + 127), fv = s.beta2 * power_of_two(ev - 30 + 127);
    float x[4], dx[4], m[4], v[4];
    floats(p, PB && !MASTER, x);
    floats(g, GB, dx);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float d = dx[j] * s.clip;
        const float mo = __int_as_float((int)(mw << (24 - 8 * j)) >> 4 & (int)0x87F00000);
        const float vo = __uint_as_float((j < 3 ? vw << (20 - 8 * j) : vw >> 4) & 0x0FF00000u);
        m[j] = __fadd_rn(__fmul_rn(mo, fm), __fmul_rn(s.rest1, d));
        v[j] = __fadd_rn(__fmul_rn(vo, fv), __fmul_rn(__fmul_rn(s.rest2, d), d));
        x[j] = updated_scaled(x[j], keep, m[j], v[j], s);
    }
    const float mt = max_nan(max_nan(fabsf(m[0]), fabsf(m[1])), max_nan(fabsf(m[2]), fabsf(m[3])));
    const float vt = max_nan(max_nan(v[0], v[1]), max_nan(v[2], v[3]));
    // exponents where a float32 has them
    constexpr uint32_t EXPONENT = 0x7F800000u, LEAST = (uint32_t)LEAST_EXPONENT << 23;
    const uint32_t me = max(__reduce_max_sync(0xffffffffu, __float_as_uint(mt)) & EXPONENT, LEAST);
    const uint32_t ve = max(__reduce_max_sync(0xffffffffu, __float_as_uint(vt)) & EXPONENT, LEAST);
    if (me > (uint32_t)MOST_M << 23 || ve > (uint32_t)MOST_V << 23) return false;
    const float sm = __uint_as_float(((14u + 127u) << 23) - me), sv = __uint_as_float(((30u + 127u) << 23) - ve);
    const uint32_t x0 = ((uint32_t)at + key) * 747796405u + 2891336453u;
    uint32_t mc[4], vc[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t h = x0 + (uint32_t)j * 747796405u;
        const uint32_t w = ((h >> ((h >> 28) + 4u)) ^ h) * 277803737u, noise = (w >> 22) ^ w;
        // the random 16 bits, and half of the next one, 4 bits up as the codes
        const uint32_t rm = __byte_perm(noise, 0x80u, 0x5104), rv = __byte_perm(noise, 0x80u, 0x5324);
        // (A funnel shift: with a plain shift of these bits, or 16 times them, this kernel's codes came out as 0.)
        mc[j] = (__funnelshift_l(0u, __float_as_uint(fabsf(m[j]) * sm), 4) + rm) | (__float_as_uint(m[j]) & 0x80000000u);
        vc[j] = __funnelshift_l(0u, __float_as_uint(v[j] * sv), 4) + rv;
        if (v[j] > 0.0f) vc[j] = max(vc[j], 1u << 24);
        if (PB) b[j] = MASTER ? round_bf16(x[j]) : round_bf16_at_random(x[j], pcg(noise) & 0xFFFFu);
    }
    if (MASTER) store_f32(it.master, at, 4, true, x);
    if (PB) store_16(it.param, at, 4, true, b);
    else store_f32(it.param, at, 4, true, x);
    auto top_bytes = [](const uint32_t (&c)[4]) { return __byte_perm(__byte_perm(c[0], c[1], 0x73), __byte_perm(c[2], c[3], 0x73), 0x5410); };
    store_codes(it.m, at, 4, true, top_bytes(mc));
    store_codes(it.v, at, 4, true, top_bytes(vc));
    if ((threadIdx.x & 31) == 0) it.scales[at / ROW] = make_uchar2((unsigned char)(me >> 23), (unsigned char)(ve >> 23));
    return true;
}

// The same for float32 moments.
template <bool PB, bool MASTER, bool GB>
__device__ __forceinline__ void row_of_32_bits(const Item& it, int64_t at, const Raw& p, const Raw& g, const Raw& mw, const Raw& vw,
                                               const Rates& s, float keep, uint32_t key)
{
    float x[4], dx[4], m[4], v[4];
    floats(p, PB && !MASTER, x);
    floats(g, GB, dx);
    floats(mw, false, m);
    floats(vw, false, v);
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float d = dx[j] * s.clip;
        m[j] = fmaf(s.beta1, m[j], s.rest1 * d);
        v[j] = fmaf(s.beta2, v[j], s.rest2 * d * d);
        x[j] = updated(x[j], keep, m[j], v[j], s);
        if (PB) b[j] = MASTER ? round_bf16(x[j]) : round_bf16_at_random(x[j], pcg(pcg((uint32_t)at + (uint32_t)j + key)) & 0xFFFFu);
    }
    if (MASTER) store_f32(it.master, at, 4, true, x);
    if (PB) store_16(it.param, at, 4, true, b);
    else store_f32(it.param, at, 4, true, x);
    store_f32(it.m, at, 4, true, m);
    store_f32(it.v, at, 4, true, v);
}

__device__ __forceinline__ Rates rates_of(const Step& a)
{
    const Clock& k = *a.clock;
    Rates s;
    s.beta1 = k.keep1, s.beta2 = k.keep2, s.rest1 = k.rest1, s.rest2 = k.rest2, s.correct2 = k.correct2;
    s.lr = a.lr_at ? __ldcg(a.lr_at) : a.lr;
    s.rate = s.lr * k.correct1;
    s.step = (uint32_t)(k.step + 1);
    s.clip = 1.0f;
    if (a.norm) {
        s.clip = a.max_norm / (__ldcg(a.norm) + 1e-6f);
        if (s.clip > 1.0f) s.clip = 1.0f;  // a NaN stays one
    }
    s.eps = a.eps;
    s.seed = a.seed;
    return s;
}

// The last block to finish a step moves its clock on.
__device__ __forceinline__ void advance(const Step& a)
{
    if (!a.last) return;
    __syncthreads();  // every thread has read the clock
    if (threadIdx.x == 0 && atomicAdd(&a.clock->finished, 1u) == gridDim.x - 1) {
        Clock& k = *a.clock;
        k.finished = 0u;
        k.step += 1;
        k.power1 *= k.beta1;
        k.power2 *= k.beta2;
        k.correct1 = (float)(1.0 / (1.0 - k.power1));
        k.correct2 = (float)(1.0 / (1.0 - k.power2));
    }
}

// The item of chunk c, from one that begins no later on.
template <int N>
__device__ __forceinline__ int item_of(const Table<N>& t, uint32_t c, int item)
{
    for (int half = N / 2; half > 0; half /= 2)
        if (item + half < t.n && t.items[item + half].chunk0 <= c) item += half;
    return item;
}

// A tensor's types, known where the code is compiled: f is called with one of these.
template <bool PB, bool MASTER, bool GB>
struct Types {
    static constexpr bool param_bf16 = PB, master = MASTER, grad_bf16 = GB;
};
template <class F>
__device__ __forceinline__ void by_types(const Item& it, F&& f)
{
    if (!it.param_bf16) it.grad_bf16 ? f(Types<false, false, true>()) : f(Types<false, false, false>());
    else if (it.master) it.grad_bf16 ? f(Types<true, true, true>()) : f(Types<true, true, false>());
    else it.grad_bf16 ? f(Types<true, false, true>()) : f(Types<true, false, false>());
}

// ---- float32 moments: a warp's ROWS rows of a chunk at once, every load first ----

constexpr int ROWS32 = 4, BLOCKS32 = 2;
template <int ROWS>
constexpr int CHUNK = ROWS * WARPS * ROW;

template <int ROWS, bool PB, bool MASTER, bool GB>
__device__ __forceinline__ void whole_rows(const Item& it, int64_t e0, const Rates& s)
{
    const uint32_t key = pcg(pcg(pcg(s.seed) + it.id) + s.step);
    const float keep = 1.0f - s.lr * it.decay;
    Raw p[ROWS], g[ROWS], m[ROWS], v[ROWS];
    const int64_t at0 = e0 + 4 * (threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t at = at0 + i * (WARPS * ROW);
        p[i] = load4(MASTER ? it.master : it.param, PB && !MASTER, at, 4, true);
        g[i] = load4(it.grad, GB, at, 4, true);
        m[i] = load4(it.m, false, at, 4, true);
        v[i] = load4(it.v, false, at, 4, true);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
        row_of_32_bits<PB, MASTER, GB>(it, at0 + i * (WARPS * ROW), p[i], g[i], m[i], v[i], s, keep, key);
}

template <int ROWS, int N>
__global__ void __launch_bounds__(THREADS, BLOCKS32) adamw_kernel(const __grid_constant__ Table<N> t, const __grid_constant__ Step a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5;
    const Rates s = rates_of(a);
    int item = 0;
    for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        item = item_of(t, c, item);
        const Item& it = t.items[item];
        const int64_t first = (int64_t)(c - it.chunk0) * CHUNK<ROWS>, e0 = first + warp * ROW;  // row i: WARPS * ROW further on
        if (it.vectors && first + CHUNK<ROWS> <= it.numel) {
            by_types(it, [&](auto types) {
                using T = decltype(types);
                whole_rows<ROWS, T::param_bf16, T::master, T::grad_bf16>(it, e0, s);
            });
        } else {
            for (int64_t row = e0; row < min(first + CHUNK<ROWS>, it.numel); row += WARPS * ROW) any_row<false>(it, row, s);
        }
    }
    advance(a);
}

// ---- 8-bit moments ----
// A warp takes strips of STRIP rows in turn, and the next strip's values come into shared
// memory (cp.async) while it computes one: the arithmetic, 74 instructions an element,
// leaves no registers for loads that far ahead, and without them a warp waited 2.7 us for
// its rows (50 M elements: 188 us, issue slots 53 % busy). A lane copies and reads its own
// elements only, so nothing is synchronised.

constexpr int STRIP8 = 4, THREADS8 = 64, WARPS8 = THREADS8 / 32, BLOCKS8 = 10;

template <int BYTES>
__device__ __forceinline__ void copy_async(void* shared, const void* global)
{
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(shared);
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(global) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(global), "n"(BYTES) : "memory");
}
// 4 elements of float32 or bf16
__device__ __forceinline__ void copy_async4(void* shared, const void* global, bool bf16, int64_t at)
{
    if (bf16) copy_async<8>(shared, static_cast<const char*>(global) + 2 * at);
    else copy_async<16>(shared, static_cast<const char*>(global) + 4 * at);
}

template <int STRIP, int N>
__global__ void __launch_bounds__(THREADS8, BLOCKS8) adamw8_kernel(const __grid_constant__ Table<N> t, const __grid_constant__ Step a)
{
    __shared__ uint4 sp[2][STRIP][THREADS8], sg[2][STRIP][THREADS8];
    __shared__ uint32_t sm[2][STRIP][THREADS8], sv[2][STRIP][THREADS8];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int me = (int)threadIdx.x, lane = me & 31;
    const Rates s = rates_of(a);
    struct Strip {
        int item, rows;    // rows that are whole and aligned
        int64_t e0;        // first element
        uint32_t scales;   // lane i: the exponents of row i
    };
    auto fetch = [&](uint32_t c, int item, int buf) {
        Strip n;
        n.item = item_of(t, c, item);
        const Item& it = t.items[n.item];
        n.e0 = (int64_t)(c - it.chunk0) * (STRIP * ROW);
        n.rows = it.vectors ? (int)min((it.numel - n.e0) / ROW, (int64_t)STRIP) : 0;
        n.scales = 0u;
        if (lane < n.rows) {
            const uchar2 e = __ldcs(it.scales + n.e0 / ROW + lane);
            n.scales = (uint32_t)e.x | (uint32_t)e.y << 8;
        }
#pragma unroll
        for (int i = 0; i < STRIP; ++i) {
            if (i >= n.rows) break;
            const int64_t at = n.e0 + i * ROW + 4 * lane;
            if (it.master) copy_async4(&sp[buf][i][me], it.master, false, at);
            else copy_async4(&sp[buf][i][me], it.param, it.param_bf16, at);
            copy_async4(&sg[buf][i][me], it.grad, it.grad_bf16, at);
            copy_async<4>(&sm[buf][i][me], static_cast<const char*>(it.m) + at);
            copy_async<4>(&sv[buf][i][me], static_cast<const char*>(it.v) + at);
        }
        return n;
    };
    const uint32_t stride = gridDim.x * WARPS8;
    uint32_t c = blockIdx.x * WARPS8 + (uint32_t)(me >> 5);
    int buf = 0;
    Strip now = {0, 0, 0, 0u}, next = now;
    if (c < t.chunks) now = fetch(c, 0, 0);
    asm volatile("cp.async.commit_group;" ::: "memory");
    for (; c < t.chunks; c += stride) {
        if (c + stride < t.chunks) next = fetch(c + stride, now.item, buf ^ 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        const Item& it = t.items[now.item];
        by_types(it, [&](auto types) {
            using T = decltype(types);
            const uint32_t key = pcg(pcg(pcg(s.seed) + it.id) + s.step);
            const float keep = 1.0f - s.lr * it.decay;
#pragma unroll 1
            for (int i = 0; i < now.rows; ++i) {
                const uint32_t e = __shfl_sync(0xffffffffu, now.scales, i);
                const int64_t row = now.e0 + i * ROW;
                if (!row_of_8_bits<T::param_bf16, T::master, T::grad_bf16>(it, row + 4 * lane, Raw{sp[buf][i][me]},
                                                                           Raw{sg[buf][i][me]}, sm[buf][i][me], sv[buf][i][me],
                                                                           make_uchar2(e & 255u, e >> 8), s, keep, key))
                    any_row<true>(it, row, s);
            }
        });
        for (int64_t row = now.e0 + now.rows * ROW; row < min(now.e0 + STRIP * ROW, it.numel); row += ROW) any_row<true>(it, row, s);
        now = next;
        buf ^= 1;
    }
    advance(a);
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

// Values of 8-bit moments: 8 elements a thread, 16 threads a block of the format (16 a
// thread left half of every sector to another store: 61 us for 50 M elements, 49 so). Its
// dependents are not launched early: a step's blocks, which share the work evenly, would
// find some SMs taken (19 M elements, step and values in turn: 105 us, 92 so).
template <bool F32>
__global__ void __launch_bounds__(THREADS) adamw_values_kernel(const uint2* m8, const uint2* v8, const uchar2* scales, void* m,
                                                               void* v, int64_t units)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t stride = (int64_t)gridDim.x * THREADS;
#pragma unroll 4
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < units; i += stride) {
        const uchar2 sc = scales[i / (ROW / 8)];
        const float ms = block_scale(sc.x, 134), vs = block_scale(sc.y, 142);
        const uint2 a = __ldcs(m8 + i), b = __ldcs(v8 + i);
        float x[8], y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = decode_m((j < 4 ? a.x : a.y) >> 8 * (j % 4) & 255u, ms);
            y[j] = decode_v((j < 4 ? b.x : b.y) >> 8 * (j % 4) & 255u, vs);
        }
        if constexpr (F32) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                __stcs(static_cast<float4*>(m) + 2 * i + q, make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]));
                __stcs(static_cast<float4*>(v) + 2 * i + q, make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]));
            }
        } else {
            uint32_t p[4], q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                p[j] = round_bf16(x[2 * j]) | round_bf16(x[2 * j + 1]) << 16;
                q[j] = round_bf16(y[2 * j]) | round_bf16(y[2 * j + 1]) << 16;
            }
            __stcs(static_cast<uint4*>(m) + i, make_uint4(p[0], p[1], p[2], p[3]));
            __stcs(static_cast<uint4*>(v) + i, make_uint4(q[0], q[1], q[2], q[3]));
        }
    }
}

// ---- host side --------------------------------------------------------------------

// Table by table, in chunks of `chunk` elements. The step's clock moves on with the last
// one, which runs (on one block) even when there is nothing to update.
template <int N>
int run(const char* fn, std::vector<Item>& items, Step s, void (*kernel)(Table<N>, Step), int64_t chunk, int threads,
        int chunks_of_block, int blocks, cudaStream_t stream)
{
    static thread_local Table<N> t;
    size_t i = 0;
    do {
        t.n = 0;
        uint64_t chunks = 0;
        for (; i < items.size() && t.n < N; ++i) {
            const uint64_t add = ((uint64_t)items[i].numel + chunk - 1) / chunk;
            if (t.n > 0 && chunks + add > 0x7fffffffu) break;
            items[i].chunk0 = (uint32_t)chunks;
            t.items[t.n++] = items[i];
            chunks += add;
        }
        t.chunks = (uint32_t)chunks;
        s.last = i >= items.size();
        const uint64_t wanted = (chunks + chunks_of_block - 1) / chunks_of_block;
        const int st = launch(fn, kernel, (unsigned)std::max<uint64_t>(1, std::min<uint64_t>(wanted, (uint64_t)blocks)), threads,
                              stream, t, s);
        if (st) return st;
    } while (i < items.size());
    return RTP_OK;
}

// One row a warp and chunk where more would leave warps without any.
template <int N>
int run_sized(const char* fn, std::vector<Item>& items, uint64_t elements, int bits, const Step& s, int sms, cudaStream_t stream)
{
    if (bits == 8) {
        const int blocks = sms * BLOCKS8;
        if (elements < (uint64_t)blocks * WARPS8 * STRIP8 * ROW)
            return run<N>(fn, items, s, adamw8_kernel<1, N>, ROW, THREADS8, WARPS8, blocks, stream);
        return run<N>(fn, items, s, adamw8_kernel<STRIP8, N>, STRIP8 * ROW, THREADS8, WARPS8, blocks, stream);
    }
    const int blocks = sms * BLOCKS32;
    if (elements < (uint64_t)blocks * CHUNK<ROWS32>)
        return run<N>(fn, items, s, adamw_kernel<1, N>, CHUNK<1>, THREADS, 1, blocks, stream);
    return run<N>(fn, items, s, adamw_kernel<ROWS32, N>, CHUNK<ROWS32>, THREADS, 1, blocks, stream);
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
        if (w.numel < 0 || w.numel >= (int64_t)1 << 39) return fail(RTP_ESHAPE, "%s: tensor %d has %lld elements", fn, i, (long long)w.numel);
        if (!(w.weight_decay >= 0.0f)) return fail(RTP_EINVAL, "%s: weight decay %g of tensor %d is not a number >= 0", fn, (double)w.weight_decay, i);
        if (w.noise < 0) return fail(RTP_EINVAL, "%s: noise %d of tensor %d is below 0", fn, w.noise, i);
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
                   w.weight_decay, (uint32_t)(w.noise ? w.noise - 1 : i), pb, gb, (uint8_t)(!(f32s & 15u) && !(b16s & 7u) && !(b8s & 3u)), 0};
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
    return items.size() <= SMALL ? run_sized<SMALL>(fn, items, elements, bits, s, sms, stream)
                                 : run_sized<LARGE>(fn, items, elements, bits, s, sms, stream);
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
    const int64_t units = blocks * (ROW / 8);
    const unsigned grid = (unsigned)std::min<int64_t>((units + THREADS - 1) / THREADS, (int64_t)sms * 8);
    return launch(fn, dtype == RTP_F32 ? adamw_values_kernel<true> : adamw_values_kernel<false>, grid, THREADS,
                  static_cast<cudaStream_t>(stream), reinterpret_cast<const uint2*>(exp_avg),
                  reinterpret_cast<const uint2*>(exp_avg_sq), reinterpret_cast<const uchar2*>(scales), m, v, units);
}

}  // extern "C"
