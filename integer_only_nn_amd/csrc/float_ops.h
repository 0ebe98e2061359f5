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
// Phi(z) = sigmoid(z Q(z^2)) with Q the polynomial that comes nearest to
// logit(Phi(z)) / z (a least-maximum fit, weighted by z Phi (1 - Phi), over z
// in (0, 6.5]; it stays positive and grows beyond).  It keeps the negative
// tail's scale, where 1 + erf cancels, and takes 10 or 13 instructions, two of
// them quarter-rate, where erfc takes about 40; the passes over 8192 x 4096
// values are bound by them.
//   8 terms: off by at most 1.2e-7, two half steps of float32 at 1, which the
//     rounding of the argument leaves anyway;
//   5 terms: 1.5e-6, a hundredth of half a step of bfloat16 at 1, for values
//     that are rounded to 16 bits.  Not for derivatives: their column sums
//     are float32, and the fit's error does not average out in them.
constexpr int kTermsGrad = 8;
template <class T>
constexpr int kTermsValue = sizeof(T) == 4 ? 8 : 5;

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kGeluK = 1.59576912160573071f;  // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;
constexpr float kLog2InvSqrt2Pi = -1.32574806473616f;  // log2(1 / sqrt(2 pi))

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// 1 / (1 + 2^x): the logistic function of -x ln 2
__device__ __forceinline__ float logistic2(float x) { return __builtin_amdgcn_rcpf(1.0f + exp2_fast(x)); }
// The factor z of a product with a vanishing one, kept finite: the limits at
// z = -inf (0) and, in the derivatives, at +inf (1) come out instead of
// inf * 0.  A NaN passes through the other factor.
__device__ __forceinline__ float above(float z) { return fmaxf(z, -200.0f); }
__device__ __forceinline__ float within(float z) { return __builtin_amdgcn_fmed3f(z, -30.0f, 30.0f); }

// Phi(z), u = z^2.
template <int TERMS>
__device__ __forceinline__ float normal_cdf(float z, float u) {
    constexpr float c8[8] = {1.5957697844099097e+00f, 7.266674921058917e-02f,  -6.60603328097877e-05f, -1.1009835059468343e-04f,
                             7.788852044459863e-06f,  -2.45761265691951e-07f, 2.3421368291093768e-09f, 2.696477063689756e-11f};
    constexpr float c5[5] = {1.59573911e+00f, 7.27856189e-02f, -1.76439094e-04f, -7.32000513e-05f, 2.83706209e-06f};
    float q = -kLog2e * (TERMS == 8 ? c8[7] : c5[4]);
#pragma unroll
    for (int i = TERMS - 2; i >= 0; --i) q = fmaf(q, u, -kLog2e * (TERMS == 8 ? c8[i] : c5[i < 5 ? i : 4]));
    return logistic2(z * q);
}

template <int ACT, int TERMS>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == IONN_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if (ACT == IONN_ACT_GELU) return above(z) * normal_cdf<TERMS>(z, z * z);
    if (ACT == IONN_ACT_GELU_TANH)
        return above(z) * logistic2(z * fmaf(z * z, -kLog2e * kGeluK * kGeluC, -kLog2e * kGeluK));
    if (ACT == IONN_ACT_SILU) return above(z) * logistic2(-kLog2e * z);
    return z;
}

template <int ACT, int TERMS>
__device__ __forceinline__ float act_grad(float z) {
    if (ACT == IONN_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    if (ACT == IONN_ACT_GELU) {  // Phi + z phi
        const float u = z * z;
        return fmaf(within(z), exp2_fast(fmaf(u, -0.5f * kLog2e, kLog2InvSqrt2Pi)), normal_cdf<TERMS>(z, u));
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
