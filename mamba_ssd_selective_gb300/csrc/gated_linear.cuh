// Shared device code of the gated linear recurrence and of values held in 8 bits:
// vectors of V channels, the gates of a token, and the conversion to 8 bits.
#pragma once
#include "common.cuh"

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

// float32 inputs take expf; bf16 inputs, whose results are rounded to 8 bits, the exponential of the special function unit (2 units
// in the last place, and that of its argument: 1e-6 relative at |x| = 8).
template <typename T> __device__ __forceinline__ float exp_of(float x) {
    if constexpr (sizeof(T) == 4) return expf(x);
    return __expf(x);
}

__device__ __forceinline__ float rsqrt_approx(float x) {
    float r;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 - exp(-2 w), a = exp(-w). Where 1 - a^2 would cancel (2 w < 1/2) by its series to the seventh term (the next is below
// 2e-7 of it); above, the difference of 1 and a^2 <= 0.61 costs 5e-7 at most.
__device__ __forceinline__ float one_minus_a2(float w, float a) {
    const float t = 2.f * w;
    float p = fmaf(t, 1.f / 5040.f, -1.f / 720.f);
    p = fmaf(t, p, 1.f / 120.f);
    p = fmaf(t, p, -1.f / 24.f);
    p = fmaf(t, p, 1.f / 6.f);
    p = fmaf(t, p, -0.5f);
    p = fmaf(t, p, 1.f);
    return t < 0.5f ? t * p : fmaf(-a, a, 1.f);
}

// The gates of one token and channel: rho and iota the sigmoids, w = k rho, a = exp(-w), beta = sqrt(1 - a^2).
struct Gates {
    float rho, iota, w, a, beta2, rbeta;  // rbeta = 1 / beta; beta = beta2 rbeta, 0 where w is
};
template <typename T> __device__ __forceinline__ Gates gates(float r, float i, float k) {
    Gates g;
    g.rho = rcp_approx(1.f + exp_of<T>(-r));
    g.iota = rcp_approx(1.f + exp_of<T>(-i));
    g.w = k * g.rho;
    g.a = exp_of<T>(-g.w);
    g.beta2 = one_minus_a2(g.w, g.a);
    g.rbeta = rsqrt_approx(fmaxf(g.beta2, 1e-37f));
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
// The whole number nearest to x 2^-e, as a byte: the sum with 1.5 2^23 has it in its last bits. 0 in a group that is not finite.
struct To8 {
    float inv;
    uint32_t mask;
    __device__ __forceinline__ explicit To8(uint32_t code = 0) : inv(inverse_scale(code)), mask(code == 255u ? 0u : 0xffu) {}
    __device__ __forceinline__ int8_t operator()(float x) const {
        return (int8_t)(__float_as_uint(fmaf(x, inv, 12582912.f)) & mask);
    }
};

}  // namespace linear
}  // namespace ssd
