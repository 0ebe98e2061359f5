// AdamW over many tensors in one launch per 60 of them, with float32 master
// weights and the two moments held in float32 or in 8 bits ("Mixed Precision
// Training of Convolutional Neural Networks using Integer Operations",
// section 4: the weight update runs in floating point, on FP32 weights).
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   P = P (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v / (1 - b2^t)) + eps)
//
// Bound by HBM: per weight it reads P, g, m, v and writes P, m, v, 28 bytes
// with float32 states and a float32 gradient, 12 + 1/64 + the gradient's
// with 8-bit ones and 2 more with their remainders.  A wavefront takes four or
// two chunks of 256 weights, a lane four consecutive ones of each, so that
// every access is a contiguous run and a chunk is one 8-bit block: its largest
// magnitude is a reduction inside the wavefront, and no state is read twice.
// Measured: 67.1 M weights with bfloat16 gradients and float32 states 324 us
// (1745 MB, 5.4 TB/s; a 1 GiB copy reaches 5.2), 8-bit states 184 us (940 MB, 5.1
// TB/s), with remainders 226 us (1075 MB, 4.8 TB/s: about 140 instructions per
// weight, of which the two exact roots and the division are 50, take as long as
// the bytes); 20 tensors of 268 k weights with float32 states 6.2 us, one launch.
//
// 8-bit states are E4M3 codes with one power-of-two exponent per block of
// 256.  The second moment is kept as its root r = sqrt(v): E4M3 spans 2^18
// from its smallest to its largest value, so the root covers 2^36 of v inside
// a block, and the step needs the root anyway.
//
// A step changes r by far less than the distance of two codes (at b2 = 0.999
// it falls by at most 1 part in 2000; codes are 1 in 16 to 1 in 8 apart), so
// rounding r to the nearest code would hold it where it is: after 2000 steps
// of unit gradients at 0.375 of its value, and for good where gradients shrink.
// Instead it goes to the code below or above, by a hash of the step and the
// element's index, with the probabilities that keep the expectation of v,
// which is linear in what came before.  v is then right on average and r
// scatters by about 15% around its 32-bit value (25% while it falls at b2 =
// 0.95).  With remainders, a byte more per weight, the step itself reads codes
// that are the nearest ones, at most half a code's step off, and the remainder,
// in 254ths of that step and rounded up or down like the codes above, keeps what
// they leave for the next ones: code and remainder together stay within about 2% of
// the 32-bit root, 0.5% in the mean square.
//
// The mean m leaves a code's surroundings (5.6% of the value, at most) by itself
// where a step takes more than that of it, up to b1 = 15/16, and goes to the
// nearest code.  Above, it would stay where it is once the gradients vanish
// (at b1 = 0.95 for good, at any size), and is rounded up or down as well.
#include "float_ops.h"

namespace ionn {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 60;                                   // tensors per launch (their table is an argument: 4 KiB)
static_assert(IONN_ADAMW_BLOCK == 256, "a block is 64 lanes of four weights");

// How the moments are held: float32, codes, codes with the root's remainder.
enum States { WORDS, CODES, CARRIED };

// Chunks of 256 weights per wavefront.  The 8-bit states' arithmetic takes
// nearly as long as their bytes, and overlaps them better from more and
// smaller wavefronts: with 4, 2 and 1 chunks 231, 223 and 213 us (remainders, 67.1
// M weights), but 244, 241 and 253 where each wavefront also forms the factors
// from a count on the device.
constexpr int chunks_of(int states) { return states == WORDS ? 4 : 2; }
constexpr int elems_of_wave(int states) { return chunks_of(states) * IONN_ADAMW_BLOCK; }
constexpr int elems_of_group(int states) { return elems_of_wave(states) * (kThreads / 64); }

struct Table {
    float *P[kTable];
    const void *G[kTable];
    void *M[kTable], *V[kTable];
    int8_t *S[kTable], *R[kTable];
    int64_t n[kTable];
    int32_t first[kTable + 1];  // first workgroup of each tensor; first[L] = grid size
    int32_t L;
};

// Everything about the step that is the same for every weight.
struct Hyper {
    double lr, beta1, beta2, eps, wd;
    int64_t t;
    const int32_t *step;
    const float *lr_dev, *grad_scale;
    uint32_t *absmax;
};

struct Factors {
    float b1, c1, b2, c2, rs2, eps, decay, size, scale;
    uint32_t seed;  // the step's part of the rounding's hash
    int spread;     // the mean's codes are rounded up or down by it
};

// b^t by repeated squaring, the same operations on the host and the device.
__host__ __device__ inline double ipow(double b, uint64_t t) {
#pragma clang fp contract(off)
    double r = 1.0;
    for (; t; t >>= 1, b = b * b)
        if (t & 1) r = r * b;
    return r;
}

__host__ __device__ inline Factors make_factors(const Hyper &h, int64_t t, double lr) {
#pragma clang fp contract(off)
    Factors f;
    f.b1 = float(h.beta1);
    f.c1 = float(1.0 - h.beta1);
    f.b2 = float(h.beta2);
    f.c2 = float(1.0 - h.beta2);
    f.rs2 = float(1.0 / __builtin_sqrt(1.0 - ipow(h.beta2, uint64_t(t))));
    f.eps = float(h.eps);
    f.decay = float(1.0 - lr * h.wd);
    f.size = float(lr / (1.0 - ipow(h.beta1, uint64_t(t))));
    f.scale = 1.0f;
    f.seed = uint32_t(t) * 0x6C8E9CF5u;
    f.spread = h.beta1 > 0.9375;
    return f;
}

// One weight: p, m and v (or, ROOT, r = sqrt(v) on entry in v's place) are
// updated; r returns sqrt of the new v.  No operation is fused with another.
__device__ __forceinline__ void step_one(const Factors &f, float g, float &p, float &m, float &v, float &r) {
#pragma clang fp contract(off)
    m = f.b1 * m + f.c1 * g;
    v = f.b2 * v + (f.c2 * g) * g;
    r = sqrtf(v);
    const float u = m / (r * f.rs2 + f.eps);
    p = p * f.decay - f.size * u;
}

// The root of v's next value.
__device__ __forceinline__ float next_root(const Factors &f, float g, float v) {
#pragma clang fp contract(off)
    v = f.b2 * v + (f.c2 * g) * g;
    return sqrtf(v);
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }  // e in [-126, 127]

// A number that orders as the exponents of blocks whose largest magnitude is x
// = f 2^q do (0: an all-zero block; the addition carries where f > 1.75), and the
// exponent that it stands for.
__device__ __forceinline__ uint32_t exponent_key(float x) {
    const uint32_t bits = __float_as_uint(x);
    return ((bits + 0x1fffffu) >> 23) + min(bits, 1u);
}
__device__ __forceinline__ int block_exponent(uint32_t key) { return key == 0u ? 0 : max(int(key) - 136, -126); }

__device__ __forceinline__ bool finite(float x) { return mag_bits(x) < 0x7f800000u; }

// Four E4M3 codes of a dword as floats, and back (to nearest even; the values
// are within the format's range; where some may not be finite, those become
// code 0x7f).
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
    typedef float v2f __attribute__((ext_vector_type(2)));
    const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
    x[0] = lo.x;
    x[1] = lo.y;
    x[2] = hi.x;
    x[3] = hi.y;
}

__device__ __forceinline__ uint32_t encode4(const float (&x)[4], bool all_finite) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
    if (!all_finite) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!finite(x[i])) w = (w & ~(0xff << (8 * i))) | 0x7f << (8 * i);
    }
    return uint32_t(w);
}

// Numbers of (0, 1), in steps of 2^-16, for the four weights of index 4 i .. at a
// step: a mix of the two (multiplications by odd numbers and shifts, each a
// bijection; a multiplication takes four times an addition's time, so four
// weights share them: a hash for each took 8 us more of 230 for 67.1 M weights).
__device__ __forceinline__ void draw4(uint32_t i, uint32_t seed, float (&u)[4]) {
    uint32_t h = i * 0x9E3779B9u + seed;
    h ^= h >> 16;
    h *= 0x5B8D2E35u;
    h ^= h >> 15;
    h *= 0xC6A4F30Bu;
    const uint32_t a = h ^ (h >> 16);
    h = a * 0x2D9A73E7u;
    const uint32_t b = h ^ (h >> 15);
    u[0] = (float(a & 0xffffu) + 0.5f) * 0x1p-16f;
    u[1] = (float(a >> 16) + 0.5f) * 0x1p-16f;
    u[2] = (float(b & 0xffffu) + 0.5f) * 0x1p-16f;
    u[3] = (float(b >> 16) + 0.5f) * 0x1p-16f;
}

// The distance of the E4M3 values from the one at or below a in [0, 448] to
// the next, a power of two, and its reciprocal.
struct Grid {
    float step, inverse;
};
__device__ __forceinline__ Grid grid_of(float a) {
    const uint32_t e = max(__float_as_uint(a) & 0x7f800000u, 121u << 23);  // (2^-9 apart below 2^-6)
    return Grid{__uint_as_float(e - (3u << 23)), __uint_as_float((257u << 23) - e)};
}

// The E4M3 value below or above s, above with probability (s^2 - lo^2) / (hi^2 - lo^2).
__device__ __forceinline__ float round_root(float s, float u) {
#pragma clang fp contract(off)
    const Grid g = grid_of(s);
    const float lo = floorf(s * g.inverse) * g.step;
    return (s - lo) * (s + lo) > u * (g.step * (lo + lo + g.step)) ? lo + g.step : lo;
}

// The E4M3 value on either side of s, the farther from 0 with probability (|s| - lo) / (hi - lo).
__device__ __forceinline__ float round_mean(float s, float u) {
#pragma clang fp contract(off)
    const float a = fabsf(s);
    const Grid g = grid_of(a);
    const float lo = floorf(a * g.inverse) * g.step;
    return copysignf(a - lo > u * g.step ? lo + g.step : lo, s);
}

// Remainders of roots, in 254ths of the step at the code's value c (both ends
// of a code's range, half a step away, are whole numbers, so that a root that
// drifts reaches the next code).
__device__ __forceinline__ float add_rest(float c, int rest) {
#pragma clang fp contract(off)
    return c + float(rest) * grid_of(c).step * (1.0f / 254.0f);
}
__device__ __forceinline__ int rest_of(float s, float c, float u) {
#pragma clang fp contract(off)
    const float x = floorf((s - c) * (grid_of(c).inverse * 254.0f) + u);
    return int(__builtin_amdgcn_fmed3f(x, -127.0f, 127.0f));
}

// Both halves' largest over the wavefront.
typedef uint16_t v2h __attribute__((ext_vector_type(2)));
__device__ __forceinline__ v2h wave_max(v2h v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v = __builtin_elementwise_max(v, __builtin_bit_cast(v2h, __shfl_xor(__builtin_bit_cast(int, v), off, 64)));
    return v;
}

// Four bytes at any address, the first `valid` of them.
__device__ __forceinline__ uint32_t load4(const uint8_t *p, int valid) {
    if (valid >= 4) return *reinterpret_cast<const __attribute__((aligned(1))) uint32_t *>(p);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (i < valid) w |= uint32_t(p[i]) << (8 * i);
    return w;
}

__device__ __forceinline__ void store4(uint8_t *p, uint32_t w, int valid) {
    if (valid >= 4) {
        *reinterpret_cast<__attribute__((aligned(1))) uint32_t *>(p) = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (i < valid) p[i] = uint8_t(w >> (8 * i));
}


template <class T, int STATES>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Table tab, Hyper h, Factors f) {
    constexpr bool Q8 = STATES != WORDS;
    constexpr int kChunks = chunks_of(STATES), kWaveElems = elems_of_wave(STATES);
    int l = 0;
    while (l + 1 < tab.L && int(blockIdx.x) >= tab.first[l + 1]) ++l;
    const int64_t n = tab.n[l];
    const int lane = threadIdx.x & 63;
    const int64_t w0 = int64_t(int(blockIdx.x) - tab.first[l]) * elems_of_group(STATES) + int64_t(threadIdx.x >> 6) * kWaveElems;
    float *__restrict__ P = tab.P[l];
    const T *__restrict__ G = static_cast<const T *>(tab.G[l]);
    float *M = static_cast<float *>(tab.M[l]), *V = static_cast<float *>(tab.V[l]);
    uint8_t *M8 = static_cast<uint8_t *>(tab.M[l]), *V8 = static_cast<uint8_t *>(tab.V[l]);
    int8_t *S = tab.S[l];
    uint8_t *R8 = reinterpret_cast<uint8_t *>(tab.R[l]);
    typename Vec<float, 4>::type p[kChunks], m[kChunks], v[kChunks];
    typename Vec<T, 4>::type g[kChunks];
    uint32_t mw[kChunks], vw[kChunks], rw[kChunks];
    int em[kChunks], ev[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int64_t i = w0 + c * 256 + lane * 4;
        const int valid = i < n ? int(n - i < 4 ? n - i : 4) : 0;
        p[c] = load_raw<float, 4>(P + i, valid);
        g[c] = load_raw<T, 4>(G + i, valid);
        if (Q8) {
            mw[c] = load4(M8 + i, valid);
            vw[c] = load4(V8 + i, valid);
            if (STATES == CARRIED) rw[c] = load4(R8 + i, valid);
            const int64_t b = w0 / 256 + c;
            em[c] = valid > 0 ? S[2 * b] : 0;
            ev[c] = valid > 0 ? S[2 * b + 1] : 0;
        } else {
            m[c] = load_raw<float, 4>(M + i, valid);
            v[c] = load_raw<float, 4>(V + i, valid);
        }
    }
    if (h.step || h.lr_dev) f = make_factors(h, h.step ? int64_t(*h.step) : h.t, h.lr_dev ? double(*h.lr_dev) : h.lr);
    const float scale = h.grad_scale ? *h.grad_scale : 1.0f;
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int64_t i = w0 + c * 256 + lane * 4;
        if (w0 + c * 256 >= n) break;  // the same for the whole wavefront
        const int valid = i < n ? int(n - i < 4 ? n - i : 4) : 0;
        float pn[4], mn[4], vn[4], rn[4], wn[4];  // (wn: the root with its remainder, squared; then new)
        if (Q8) {
            decode4(mw[c], mn);
            decode4(vw[c], vn);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mn[e] *= pow2f(em[c]);
                if (STATES == CARRIED) {
                    const float w = add_rest(vn[e], int8_t(rw[c] >> (8 * e))) * pow2f(ev[c]);
                    wn[e] = w * w;
                }
                const float r = vn[e] * pow2f(ev[c]);
                vn[e] = r * r;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            pn[e] = p[c][e];
            if (!Q8) {
                mn[e] = m[c][e];
                vn[e] = v[c][e];
            }
            step_one(f, float(g[c][e]) * scale, pn[e], mn[e], vn[e], rn[e]);
            wn[e] = STATES == CARRIED ? next_root(f, float(g[c][e]) * scale, wn[e]) : rn[e];
            if (e < valid) top = max(top, mag_bits(pn[e]));
        }
        store_vec<float, 4>(P + i, pn, valid);
        if (Q8) {
            // the block's largest finite magnitudes (past the tensor's end both
            // moments are 0, and a maximum with a NaN is the other value)
            float am = 0.0f, av = 0.0f;
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                am = fmaxf(am, fabsf(mn[e]));
                av = fmaxf(av, wn[e]);
                odd |= !finite(mn[e] + wn[e]);
            }
            const bool all_finite = __builtin_amdgcn_ballot_w64(odd) == 0;
            if (!all_finite) {
                am = av = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    am = fmaxf(am, finite(mn[e]) ? fabsf(mn[e]) : 0.0f);
                    av = fmaxf(av, finite(wn[e]) ? wn[e] : 0.0f);
                }
            }
            const v2h keys = wave_max(v2h{uint16_t(exponent_key(am)), uint16_t(exponent_key(av))});
            const int xm = block_exponent(keys.x), xv = block_exponent(keys.y);
            float sm[4], sv[4], u[4];
            draw4(uint32_t(i >> 2), f.seed, u);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sm[e] = mn[e] * pow2f(-xm);
                const bool positive = wn[e] > 0.0f;
                wn[e] *= pow2f(-xv);
                sv[e] = STATES == CODES ? round_root(wn[e], u[e]) : wn[e];
                // a positive root keeps at least the smallest code, 2^-9
                if (positive && sv[e] < 0x1p-9f) sv[e] = 0x1p-9f;
            }
            if (f.spread) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sm[e] = round_mean(sm[e], u[e ^ 2]);
            }
            const uint32_t codes = encode4(sv, all_finite);
            store4(M8 + i, encode4(sm, all_finite), valid);
            store4(V8 + i, codes, valid);
            if (STATES == CARRIED) {
                decode4(codes, sv);
                uint32_t w = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t q = uint32_t(rest_of(wn[e], sv[e], u[e])) & 0xffu;
                    w |= (all_finite || finite(wn[e]) ? q : 0u) << (8 * e);
                }
                store4(R8 + i, w, valid);
            }
            if (lane == 0) {
                const int64_t b = w0 / 256 + c;
                S[2 * b] = int8_t(xm);
                S[2 * b + 1] = int8_t(xv);
            }
        } else {
            store_vec<float, 4>(M + i, mn, valid);
            store_vec<float, 4>(V + i, vn, valid);
        }
    }
    if (h.absmax) {
        top = wave_max_u32(top);
        if (lane == 0) publish_max_u32(h.absmax + l, top);
    }
}

}  // namespace
}  // namespace ionn

using namespace ionn;

// (`what`: the entry point, for its messages; R NULL: no remainders)
static int adamw(const char *what, int L, float *const *P, const void *const *G, int g_dtype, void *const *M,
                 void *const *V, int8_t *const *S, int8_t *const *R, int state_bits, const int64_t *n, int64_t t,
                 double lr, double beta1, double beta2, double eps, double weight_decay, const int32_t *step,
                 const float *lr_dev, const float *grad_scale, uint32_t *absmax_P, void *stream) {
    clear_error();
    IONN_REQUIRE(L >= 1, IONN_ERR_SHAPE, "%s: L = %d < 1", what, L);
    IONN_REQUIRE(dtype_ok(g_dtype), IONN_ERR_ARG, "%s: g_dtype = %d", what, g_dtype);
    IONN_REQUIRE(state_bits == 32 || state_bits == 8, IONN_ERR_ARG, "%s: state_bits = %d (8 or 32)", what,
                 state_bits);
    IONN_REQUIRE(P && G && M && V && n && (state_bits == 32 || S), IONN_ERR_ARG, "%s: NULL array", what);
    IONN_REQUIRE(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0, IONN_ERR_RANGE,
                 "%s: beta1 = %g, beta2 = %g outside [0, 1)", what, beta1, beta2);
    IONN_REQUIRE(eps >= 0.0 && eps <= 3.0e38 && lr >= -3.0e38 && lr <= 3.0e38 && weight_decay >= -3.0e38 &&
                     weight_decay <= 3.0e38,
                 IONN_ERR_RANGE, "%s: eps = %g, lr = %g, weight_decay = %g", what, eps, lr, weight_decay);
    IONN_REQUIRE(step || t >= 1, IONN_ERR_RANGE, "%s: t = %lld < 1", what, (long long)t);
    IONN_REQUIRE(aligned(step, 4) && aligned(lr_dev, 4) && aligned(grad_scale, 4) && aligned(absmax_P, 4),
                 IONN_ERR_ALIGN, "%s: device scalars must be 4-byte aligned", what);
    const size_t gs = dtype_size(g_dtype), ss = state_bits == 32 ? 4 : 1;
    const int64_t per = elems_of_group(state_bits == 32 ? WORDS : CODES);
    static_assert(elems_of_group(CODES) == elems_of_group(CARRIED), "one layout of the 8-bit states");
    for (int l = 0; l < L; ++l) {
        IONN_REQUIRE(n[l] >= 1 && n[l] <= per * max_groups(kThreads), IONN_ERR_SHAPE, "%s: tensor %d has n = %lld",
                     what, l, (long long)n[l]);
        IONN_REQUIRE(P[l] && G[l] && M[l] && V[l] && (state_bits == 32 || S[l]), IONN_ERR_ARG,
                     "%s: tensor %d has a NULL pointer", what, l);
        IONN_REQUIRE(aligned(P[l], 4) && aligned(G[l], gs) && aligned(M[l], ss) && aligned(V[l], ss), IONN_ERR_ALIGN,
                     "%s: tensor %d must be aligned to its element size", what, l);
    }
    Hyper h{lr, beta1, beta2, eps, weight_decay, t, step, lr_dev, grad_scale, nullptr};
    const Factors f = make_factors(h, t < 1 ? 1 : t, lr);
    hipStream_t st = as_stream(stream);
    int l = 0;
    while (l < L) {
        Table tab;
        memset(&tab, 0, sizeof(tab));
        int64_t blocks = 0;
        h.absmax = absmax_P ? absmax_P + l : nullptr;
        int k = 0;
        for (; k < kTable && l < L; ++k, ++l) {
            const int64_t b = (n[l] + per - 1) / per;
            if (blocks + b > max_groups(kThreads)) break;  // (one tensor alone never is)
            tab.P[k] = P[l];
            tab.G[k] = G[l];
            tab.M[k] = M[l];
            tab.V[k] = V[l];
            tab.S[k] = state_bits == 8 ? S[l] : nullptr;
            tab.R[k] = R ? R[l] : nullptr;
            tab.n[k] = n[l];
            tab.first[k] = int32_t(blocks);
            blocks += b;
        }
        tab.first[k] = int32_t(blocks);
        tab.L = k;
        with_dtype(g_dtype, [&](auto tag) {
            using T = decltype(tag);
            const dim3 grid{unsigned(blocks)}, block{kThreads};
            if (state_bits == 32) adamw_kernel<T, WORDS><<<grid, block, 0, st>>>(tab, h, f);
            else if (!R) adamw_kernel<T, CODES><<<grid, block, 0, st>>>(tab, h, f);
            else adamw_kernel<T, CARRIED><<<grid, block, 0, st>>>(tab, h, f);
        });
        if (int rc = check_launch(what)) return rc;
    }
    return IONN_OK;
}

extern "C" {

int ionn_adamw_step(int L, float *const *P, const void *const *G, int g_dtype, void *const *M, void *const *V,
                    int8_t *const *S, int state_bits, const int64_t *n, int64_t t, double lr, double beta1,
                    double beta2, double eps, double weight_decay, const int32_t *step, const float *lr_dev,
                    const float *grad_scale, uint32_t *absmax_P, void *stream) {
    return adamw("ionn_adamw_step", L, P, G, g_dtype, M, V, S, nullptr, state_bits, n, t, lr, beta1, beta2, eps,
                 weight_decay, step, lr_dev, grad_scale, absmax_P, stream);
}

int ionn_adamw_step_carried(int L, float *const *P, const void *const *G, int g_dtype, void *const *M, void *const *V,
                            int8_t *const *S, int8_t *const *R, const int64_t *n, int64_t t, double lr, double beta1,
                            double beta2, double eps, double weight_decay, const int32_t *step, const float *lr_dev,
                            const float *grad_scale, uint32_t *absmax_P, void *stream) {
    clear_error();
    IONN_REQUIRE(R, IONN_ERR_ARG, "ionn_adamw_step_carried: NULL array");
    for (int l = 0; l < L; ++l)
        IONN_REQUIRE(R[l], IONN_ERR_ARG, "ionn_adamw_step_carried: tensor %d has a NULL pointer", l);
    return adamw("ionn_adamw_step_carried", L, P, G, g_dtype, M, V, S, R, 8, n, t, lr, beta1, beta2, eps, weight_decay,
                 step, lr_dev, grad_scale, absmax_P, stream);
}

}  // extern "C"
