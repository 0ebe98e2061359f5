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
// Phi(z) = sigmoid(z Q(z^2)) with Q the polynomial of degree 7 that comes
// nearest to logit(Phi(z)) / z (a least-maximum fit, weighted by z Phi (1 -
// Phi), over z in (0, 6.5]; it stays positive and grows beyond).  Phi is off by
// at most 1.2e-7, two half steps of float32 at 1, which the rounding of the
// argument leaves anyway, and keeps the negative tail's scale, where 1 + erf
// cancels.  It takes 13 instructions, two of them quarter-rate, where erfc
// takes about 40 (the epilogue of an 8192 x 4096 output is bound by them).

constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kGeluK = 1.59576912160573071f;  // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;
constexpr float kLog2e = 1.44269504088896341f;

// The factor z of a product with a vanishing one, kept finite: the limits at
// z = -inf (0) and, in the derivatives, at +inf (1) come out instead of
// inf * 0.  A NaN passes through the other factor.
__device__ __forceinline__ float above(float z) { return fmaxf(z, -200.0f); }
__device__ __forceinline__ float within(float z) { return __builtin_amdgcn_fmed3f(z, -30.0f, 30.0f); }

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float sigmoid(float w) { return __builtin_amdgcn_rcpf(1.0f + exp2_fast(-kLog2e * w)); }

__device__ __forceinline__ float normal_cdf(float z) {
    constexpr float c[8] = {1.5957697844099097e+00f * -kLog2e,  7.266674921058917e-02f * -kLog2e,
                            -6.60603328097877e-05f * -kLog2e,   -1.1009835059468343e-04f * -kLog2e,
                            7.788852044459863e-06f * -kLog2e,   -2.45761265691951e-07f * -kLog2e,
                            2.3421368291093768e-09f * -kLog2e,  2.696477063689756e-11f * -kLog2e};
    const float u = z * z;
    float q = c[7];
#pragma unroll
    for (int i = 6; i >= 0; --i) q = fmaf(q, u, c[i]);
    return __builtin_amdgcn_rcpf(1.0f + exp2_fast(z * q));
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == IONN_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if (ACT == IONN_ACT_GELU) return above(z) * normal_cdf(z);
    if (ACT == IONN_ACT_GELU_TANH) return above(z) * sigmoid(kGeluK * (z + kGeluC * z * z * z));
    if (ACT == IONN_ACT_SILU) return above(z) * sigmoid(z);
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
    if (ACT == IONN_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    if (ACT == IONN_ACT_GELU) {
        const float y = within(z);
        return normal_cdf(z) + y * kInvSqrt2Pi * exp2_fast(-0.5f * kLog2e * (y * y));
    }
    if (ACT == IONN_ACT_GELU_TANH) {
        const float y = within(z);
        const float p = sigmoid(kGeluK * (z + kGeluC * z * z * z));
        return p + y * p * (1.0f - p) * (kGeluK * (1.0f + 3.0f * kGeluC * y * y));
    }
    if (ACT == IONN_ACT_SILU) {
        const float p = sigmoid(z);
        return p * (1.0f + within(z) * (1.0f - p));
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

// sat8(rne(x / 2^E)), given -E in [-121, 155].  ldexp is exact here unless
// its result is below 2^-126, which rounds to 0 as the exact one does.
__device__ __forceinline__ int32_t dfp8_mantissa(float x, int negE) {
    const float r = __builtin_rintf(__builtin_amdgcn_ldexpf(x, negE));
    return int32_t(fminf(fmaxf(r, -128.0f), 127.0f));
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
