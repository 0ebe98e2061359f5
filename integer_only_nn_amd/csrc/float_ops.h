// Floating tensors around the integer products: element types, 16-byte
// vectors, activations and their derivatives, and the reductions that the
// layer norm, DFP-8 and optimiser kernels share.  Arithmetic is in float32
// whatever the tensor's type; a value is rounded to its type once, when it is
// stored (to nearest even).
#pragma once

#include "common.h"

namespace ionn {

typedef __bf16 bf16;
typedef _Float16 f16;
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

inline bool dtype_ok(int dtype) { return dtype == IONN_F32 || dtype == IONN_BF16 || dtype == IONN_F16; }
inline size_t dtype_size(int dtype) { return dtype == IONN_F32 ? 4 : 2; }

// A grid has fewer than 2^32 threads along a dimension; the runtime takes some
// larger ones without a word and runs the rest of their division by 2^32.
constexpr int64_t max_groups(int threads) { return int64_t(0xffffffffu) / threads; }

// Calls f with a value of the element type of `dtype` (checked before).
template <class F>
inline void with_dtype(int dtype, F &&f) {
    if (dtype == IONN_F32) f(float{});
    else if (dtype == IONN_BF16) f(bf16{});
    else f(f16{});
}

// VE consecutive elements of T at any address that suits a single element (the
// hardware takes 16-byte accesses at any byte; rows of odd length start
// anywhere, so no path asks for more).
template <class T, int VE>
struct Vec {
    typedef T type __attribute__((ext_vector_type(VE)));
    typedef T loose __attribute__((ext_vector_type(VE), aligned(alignof(T))));
};

template <class T, int VE>
__device__ __forceinline__ typename Vec<T, VE>::type load_raw(const T *p) {
    return *reinterpret_cast<const typename Vec<T, VE>::loose *>(p);
}

// The first `valid` of VE elements at p, zeros after them.
template <class T, int VE>
__device__ __forceinline__ typename Vec<T, VE>::type load_raw(const T *p, int valid) {
    if (valid >= VE) return load_raw<T, VE>(p);
    typename Vec<T, VE>::type v;
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = i < valid ? p[i] : T(0.0f);
    return v;
}

template <class T, int VE>
__device__ __forceinline__ void store_vec(T *p, const float (&x)[VE], int valid = VE) {
    typename Vec<T, VE>::type v;
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = T(x[i]);
    if (valid >= VE) {
        *reinterpret_cast<typename Vec<T, VE>::loose *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < VE; ++i)
            if (i < valid) p[i] = v[i];
    }
}

// ---- activations -------------------------------------------------------------
// The value and the derivative at z.  gelu is z * Phi(z) with the normal
// distribution function Phi; gelu_tanh is z * sigmoid(2 k (z + c z^3)), k =
// sqrt(2 / pi), c = 0.044715 (0.5 (1 + tanh w) = sigmoid(2 w)).
//
// Phi's tail is Phi(-x) = exp(-x^2 / 2) t P(t), t = 1 / (1 + p x), with p and the
// polynomial P that come nearest to it in relative error over x in [0, 14] (at
// 13.2 the exponential leaves float32's range).  So gelu(z) = max(z, 0) - |z|
// Phi(-|z|) keeps its relative exactness however small it gets, where 1 + erf
// cancels.  Beside the fit's error there are the roundings of exp's argument, z^2
// half steps of float32 at most.  The passes over 8192 x 4096 values are bound by
// these instructions, two of 13 or 16 quarter-rate.
//   8 terms: off by at most 1.1e-7 of the value, two half steps of float32;
//   5 terms: 3.1e-5, a sixteenth of half a step of float16, for values that are
//     rounded to 16 bits.  Not for derivatives: their column sums are float32,
//     and the fit's error does not average out in them.
constexpr int kTermsGrad = 8;
template <class T>
constexpr int kTermsValue = sizeof(T) == 4 ? 8 : 5;

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kGeluK = 1.59576912160573071f;  // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;
constexpr float kInvSqrt2Pi = 0.398942280401432678f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// 1 / (1 + 2^x): the logistic function of -x ln 2
__device__ __forceinline__ float logistic2(float x) { return __builtin_amdgcn_rcpf(1.0f + exp2_fast(x)); }
// The factor z of a product with a vanishing one, kept finite: the limits at
// z = -inf (0) and, in the derivatives, at +inf (1) come out instead of
// inf * 0.  A NaN passes through the other factor.
__device__ __forceinline__ float above(float z) { return fmaxf(z, -200.0f); }
__device__ __forceinline__ float within(float z) { return __builtin_amdgcn_fmed3f(z, -30.0f, 30.0f); }

// exp(-x^2 / 2) and, of it, Phi(-x); x >= 0.
__device__ __forceinline__ float normal_exp(float x) { return exp2_fast(x * x * (-0.5f * kLog2e)); }
template <int TERMS>
__device__ __forceinline__ float normal_tail(float x, float e) {
    constexpr float p = TERMS == 8 ? 0.30625f : 0.375f;
    constexpr float c8[8] = {1.221450791e-01f,  1.228500903e-01f, 1.045957729e-01f,  1.180542856e-01f,
                             -3.183713555e-02f, 1.778280437e-01f, -1.501339674e-01f, 3.649786860e-02f};
    constexpr float c5[5] = {1.490610093e-01f, 1.577341557e-01f, 8.356352150e-02f, 2.002823502e-01f, -9.064312279e-02f};
    const float t = __builtin_amdgcn_rcpf(fmaf(p, x, 1.0f));
    float q = TERMS == 8 ? c8[7] : c5[4];
#pragma unroll
    for (int i = TERMS - 2; i >= 0; --i) q = fmaf(q, t, TERMS == 8 ? c8[i] : c5[i < 5 ? i : 4]);
    return e * (t * q);
}

template <int ACT, int TERMS>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == IONN_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if (ACT == IONN_ACT_GELU) {  // (|z| clipped where the tail is 0, so that infinities do not meet it)
        const float x = fabsf(z);
        return fmaf(-fminf(x, 30.0f), normal_tail<TERMS>(x, normal_exp(x)), fmaxf(z, 0.0f));
    }
    if (ACT == IONN_ACT_GELU_TANH)
        return above(z) * logistic2(z * fmaf(z * z, -kLog2e * kGeluK * kGeluC, -kLog2e * kGeluK));
    if (ACT == IONN_ACT_SILU) return above(z) * logistic2(-kLog2e * z);
    return z;
}

template <int ACT, int TERMS>
__device__ __forceinline__ float act_grad(float z) {
    if (ACT == IONN_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    if (ACT == IONN_ACT_GELU) {  // Phi + z phi
        const float x = fabsf(z), e = normal_exp(x), tail = normal_tail<TERMS>(x, e);
        return fmaf(within(z) * kInvSqrt2Pi, e, z < 0.0f ? tail : 1.0f - tail);
    }
    if (ACT == IONN_ACT_GELU_TANH) {
        const float p = logistic2(z * fmaf(z * z, -kLog2e * kGeluK * kGeluC, -kLog2e * kGeluK)), y = within(z);
        return fmaf(y * fmaf(y * y, 3.0f * kGeluK * kGeluC, kGeluK), p * (1.0f - p), p);
    }
    if (ACT == IONN_ACT_SILU) {
        const float p = logistic2(-kLog2e * z);
        return p * fmaf(within(z), 1.0f - p, 1.0f);
    }
    return 1.0f;
}

template <int V>
struct IntC {
    static constexpr int value = V;
};

// Calls f with the activation as a compile-time constant (checked before).
template <class F>
__host__ __device__ __forceinline__ void with_act(int act, F &&f) {
    if (act == IONN_ACT_RELU) f(IntC<IONN_ACT_RELU>{});
    else if (act == IONN_ACT_GELU) f(IntC<IONN_ACT_GELU>{});
    else if (act == IONN_ACT_GELU_TANH) f(IntC<IONN_ACT_GELU_TANH>{});
    else if (act == IONN_ACT_SILU) f(IntC<IONN_ACT_SILU>{});
    else f(IntC<IONN_ACT_NONE>{});
}

// ---- DFP-8 -------------------------------------------------------------------
// Magnitude bits of a float: they order as the magnitudes do, and a NaN or an
// infinity shows as bits >= 0x7f800000.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The shared exponent of 8-bit mantissas for magnitude bits m of the largest
// value f 2^q (f in [1, 2)): q - 6, so that it lands in [64, 128); 0 for an
// all-zero or not finite tensor.
__device__ __forceinline__ int dfp8_exponent(uint32_t m) {
    if (m == 0u || m >= 0x7f800000u) return 0;
    const int ex = int(m >> 23);
    return (ex > 0 ? ex - 127 : -150 + bitlen_u32(m & 0x7fffffu)) - 6;
}

// sat8(rne(x / 2^E)) in the low byte, given -E in [-121, 155]: ldexp is exact
// here unless its result is below 2^-126, which rounds to 0 as the exact one
// does, and adding 1.5 * 2^23 rounds to an integer and leaves it in the low
// bits.
__device__ __forceinline__ uint32_t dfp8_mantissa(float x, int negE) {
    return __float_as_uint(__builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(x, negE), -128.0f, 127.0f) + 12582912.0f);
}

// 0, 1 (exponent outside the signed 8-bit range), 2 (not finite).
__device__ __forceinline__ int32_t dfp8_status(uint32_t m, int E) {
    return m >= 0x7f800000u ? 2 : (E < -128 || E > 127 ? 1 : 0);
}

// ---- reductions --------------------------------------------------------------

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

}  // namespace ionn
