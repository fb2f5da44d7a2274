// Shared device code of the gated linear recurrence and of values held in 8 bits:
// vectors of V channels, the gates of a token, and the conversion to 8 bits.
#pragma once
#include "common.cuh"
#include "f32x2.cuh"

namespace ssd {
namespace linear {

constexpr int kGroup = 16;  // tokens of a channel that share a scale
constexpr int kState = 64;  // tokens between saved states

// V neighbouring elements as they lie in memory, read and written in one access: a row of D elements, D a multiple of V, starts
// at a multiple of V elements.
template <int BYTES> struct Word;
template <> struct Word<1> { using type = uint8_t; };
template <> struct Word<2> { using type = uint16_t; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<16> { using type = uint4; };
template <typename T, int V> union Raw {
    typename Word<sizeof(T) * V>::type word;
    T v[V];
    uint32_t u[(sizeof(T) * V + 3) / 4];
    __device__ Raw() : word{} {}
};

// Every value of the sequence is used once: read and written past the L1 as the first to be replaced.
template <typename T, int V> __device__ __forceinline__ Raw<T, V> load(const T *p) {
    Raw<T, V> r;
    r.word = __ldcs(reinterpret_cast<const typename Word<sizeof(T) * V>::type *>(p));
    return r;
}
template <typename T, int V> __device__ __forceinline__ void store(T *p, const Raw<T, V> &r) {
    __stcs(reinterpret_cast<typename Word<sizeof(T) * V>::type *>(p), r.word);
}
template <typename T, int V> __device__ __forceinline__ void store_f32(T *p, const float (&f)[V]) {
    Raw<T, V> r;
#pragma unroll
    for (int v = 0; v < V; ++v) r.v[v] = from_f32<T>(f[v]);
    store<T, V>(p, r);
}

// c softplus(lam), and sigmoid(lam) / softplus(lam), which turns sums over w dL/dw into the gradient of lam. Below -16 the
// first is c exp(lam) and the second 1 to 2^-23.
__device__ __forceinline__ float softplus(float lam) { return lam > 20.f ? lam : log1pf(expf(lam)); }
__device__ __forceinline__ float softplus_ratio(float lam) {
    return lam < -16.f ? 1.f : 1.f / ((1.f + expf(-lam)) * softplus(lam));
}

__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

using delta::add2;
using delta::f2;
using delta::fma2;
using delta::mul2;
using delta::un2;
__device__ __forceinline__ uint64_t f2(float x) { return f2(x, x); }
__device__ __forceinline__ uint64_t pair_of(const Raw<float, 2> &r) { return f2(r.v[0], r.v[1]); }
__device__ __forceinline__ uint64_t pair_of(const Raw<__nv_bfloat16, 2> &r) {
    return f2(__uint_as_float(r.word << 16), __uint_as_float(r.word & 0xffff0000u));
}

constexpr float kLog2e = 1.4426950408889634f, kLog2eRest = 1.9259629911e-8f, kLn2 = 0.6931471805599453f;

// exp(-x) for two numbers: within 2 units in the last place, and that of its argument (|x| 1e-7 relative). float32 inputs get
// the argument's rest too; the results of bf16 inputs are rounded to 8 bits.
template <typename T> __device__ __forceinline__ uint64_t exp_minus(uint64_t x) {
    const uint64_t y = mul2(x, f2(kLog2e));
    float y0, y1;
    un2(y, y0, y1);
    uint64_t e = f2(ex2_approx(-y0), ex2_approx(-y1));
    if constexpr (sizeof(T) == 4) {
        const uint64_t rest = fma2(x, f2(-kLog2eRest), fma2(x, f2(-kLog2e), y));
        // an exponential that is 0 or infinite stays so: its rest is finite, and with x infinite not a number
        const uint64_t f = fma2(e, mul2(rest, f2(kLn2)), e);
        float f0, f1, e0, e1;
        un2(f, f0, f1);
        un2(e, e0, e1);
        e = f2(fabsf(y0) < 126.f ? f0 : e0, fabsf(y1) < 126.f ? f1 : e1);
    }
    return e;
}

// The gates of one token, for two channels, with rho and iota the sigmoids of r and i, w = k rho and t = 2 w:
//     a = exp(-w)     f = sqrt(1 - a^2) iota     and for the backward g = a^2 w / (1 - a^2) = w / (exp(2 w) - 1) (grad_ratio).
// For t < 1 all three are polynomials of degree 4 in t, exact at 0 and through Chebyshev points on [0, 1] (their error goes to zero
// with t, and most tokens' t is small): a as 1 + t E(t) (E 5e-8 off at t = 1/5, 3.5e-7 at 1), f as sqrt(2 k rho) Q(t) iota with
// Q(t) = sqrt((1 - e^-t) / t) (9e-8, 6e-7), g as G(t) = t / (e^t - 1) / 2 (1.1e-7, 1.2e-6). So there is neither a difference that
// cancels nor a root of its own to take: rho is the square of 1 / sqrt(1 + e^-r). And a is rounded once: an a off by d counts d / w in
// h, and the approximate exponential, off by 1e-7 to one side near 1, made h 1.3e-6 wrong where this makes it 2e-7 (float32 B2 L777).
// FAST, for what nearly every run of tokens is: k below kSteep, so that t < 1, and r and i (r + 2 i above -88 or so) such that the
// argument of one reciprocal root, sqrt(rho) iota = 1 / sqrt((1 + e^-r) (1 + e^-i)^2), is finite: `sum` adds them up and tells.
// Three calls of the special function unit a token and channel instead of four, and no choice.
// The gradients of r and i have 1 - rho and 1 - iota: e^-r rho and e^-i iota, as a difference of an open gate is its error and no more
// (at r = 16 zero or negative). A gate that is zero has an infinite exponential, which counts as the largest number: the product, zero
// then, meets nothing but a zero.
constexpr float kSteep = 0.5f;
struct Rate2 {  // of two channels: 2 k, sqrt(2 k)
    uint64_t twice, root;
    __device__ __forceinline__ static Rate2 of(float k0, float k1) {
        return {f2(2.f * k0, 2.f * k1), f2(sqrtf(2.f * k0), sqrtf(2.f * k1))};
    }
};
__device__ __forceinline__ uint64_t finite2(uint64_t e) {
    float e0, e1;
    un2(e, e0, e1);
    return f2(fminf(e0, 3.402823466e38f), fminf(e1, 3.402823466e38f));
}
struct Gates2 {
    uint64_t a, f, rho, t;
    uint64_t er, not_iota;  // GRAD: e^-r, finite; 1 - iota
};
template <typename T, bool FAST, bool GRAD> __device__ __forceinline__ Gates2 gates2(uint64_t r, uint64_t i, const Rate2 &k, uint64_t &sum) {
    Gates2 o;
    const uint64_t one = f2(1.f), er = exp_minus<T>(r), ei = exp_minus<T>(i), u = add2(er, one), v = add2(ei, one);
    uint64_t z;  // sqrt(rho) iota
    uint64_t iota;
    float x0, x1;
    if constexpr (FAST) {
        const uint64_t uv = mul2(u, v), uvv = mul2(uv, v);
        sum = add2(sum, uvv);
        un2(uvv, x0, x1);
        z = f2(rsqrt_approx(x0), rsqrt_approx(x1));
        const uint64_t m = mul2(z, v);
        o.rho = mul2(m, m);
        if (GRAD) o.not_iota = mul2(mul2(z, z), mul2(uv, ei));
    } else {
        un2(u, x0, x1);
        const uint64_t m = f2(rsqrt_approx(x0), rsqrt_approx(x1));
        un2(v, x0, x1);
        iota = f2(rcp_approx(x0), rcp_approx(x1));
        o.rho = mul2(m, m), z = mul2(m, iota);
        if (GRAD) o.not_iota = mul2(finite2(ei), iota);
    }
    if (GRAD) o.er = FAST ? er : finite2(er);
    o.t = mul2(o.rho, k.twice);
    uint64_t e = fma2(o.t, f2(-0.00022097997134551406f), f2(0.002580259693786502f));
    e = fma2(o.t, e, f2(-0.0208286102861166f));
    e = fma2(o.t, e, f2(0.12499985098838806f));
    e = fma2(o.t, e, f2(-0.5f));
    uint64_t q = fma2(o.t, f2(0.000725092482753098f), f2(-0.007732587866485119f));
    q = fma2(o.t, q, f2(0.05206755921244621f));
    q = fma2(o.t, q, f2(-0.2499995082616806f));
    q = fma2(o.t, q, one);
    o.a = fma2(o.t, e, one);
    o.f = mul2(mul2(z, k.root), q);
    if constexpr (!FAST) {  // t >= 1: 1 - a^2 from a^2 <= 0.37
        float t0, t1, i0, i1, f0, f1, a0, a1;
        un2(o.t, t0, t1);
        un2(iota, i0, i1);
        un2(o.f, f0, f1);
        un2(o.a, a0, a1);
        if (!(t0 < 1.f)) a0 = ex2_approx(-0.5f * kLog2e * t0), f0 = fmaf(-a0, a0, 1.f), f0 = f0 * rsqrt_approx(f0) * i0;
        if (!(t1 < 1.f)) a1 = ex2_approx(-0.5f * kLog2e * t1), f1 = fmaf(-a1, a1, 1.f), f1 = f1 * rsqrt_approx(f1) * i1;
        o.f = f2(f0, f1), o.a = f2(a0, a1);
    }
    return o;
}
// Whether the sum of gates2's arguments says that one of them was not finite.
__device__ __forceinline__ bool is_low(uint64_t sum, bool one, bool both) {
    float s0, s1;
    un2(sum, s0, s1);
    return (one && !(s0 < 3.4e38f)) || (both && !(s1 < 3.4e38f));
}
// G(t); `steep`: where t may be 1 and more.
__device__ __forceinline__ uint64_t grad_ratio(uint64_t t, uint64_t a, bool steep) {
    uint64_t g = fma2(t, f2(-0.0006504057091660798f), f2(-3.583935904316604e-05f));
    g = fma2(t, g, f2(0.04167448729276657f));
    g = fma2(t, g, f2(-0.2500002384185791f));
    g = fma2(t, g, f2(0.5f));
    if (steep) {
        float t0, t1, a0, a1, g0, g1;
        un2(t, t0, t1);
        un2(a, a0, a1);
        un2(g, g0, g1);
        if (!(t0 < 1.f)) g0 = a0 * a0 * 0.5f * t0 * rcp_approx(fmaf(-a0, a0, 1.f));
        if (!(t1 < 1.f)) g1 = a1 * a1 * 0.5f * t1 * rcp_approx(fmaf(-a1, a1, 1.f));
        g = f2(g0, g1);
    }
    return g;
}

// 8 bits: the values of a group are whole numbers times 2^e, e the least with max |x| <= 127 2^e and e >= -127, kept as the
// byte e + 127. Every step is exact but the rounding to a whole number. 255 marks a group that held a NaN or an infinity.
// `top` is the largest |x| of the group as bits, which order like the numbers, NaN above infinity.
__device__ __forceinline__ uint32_t scale_code(uint32_t top) {
    const int e = (int)(top >> 23) - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    return top >= 0x7f800000u ? 255u : (uint32_t)max(e, 0);
}
__device__ __forceinline__ float scale_of(uint32_t code) {  // 2^e
    return code == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(code ? code << 23 : 0x400000u);
}
__device__ __forceinline__ float inverse_scale(uint32_t code) {  // 2^-e
    return code == 255u ? 0.f : __uint_as_float((254u - code) << 23);
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
// x 2^-e + 1.5 2^23 has the whole number nearest to x 2^-e in its last bits.
constexpr float kToWhole = 12582912.f;

}  // namespace linear
}  // namespace ssd
