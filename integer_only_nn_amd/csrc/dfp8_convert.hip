// Conversion of floating tensors to DFP-8 (8-bit mantissas, one shared
// exponent from the exponent of the largest magnitude: "Mixed Precision
// Training of Convolutional Neural Networks using Integer Operations", 3.1),
// and the same behind an activation's derivative, where a Linear layer's
// error becomes the operand of its gradients.
//
// The exponent needs the maximum of the whole tensor before the first value
// is rounded, so both are two passes, bound by HBM: one that leaves each
// workgroup's maximum (and the error's column sums), one that rounds.  The
// second pass computes the derivative again rather than read it back: a
// float32 copy would cost 8 bytes per element where dY and Z cost 4 in the
// 16-bit types.  Each workgroup of it reduces the first pass's maxima itself
// (about 4 KiB, from L2), which saves the launch, the cleared scalar and the
// queue of atomics of a shared maximum.  8192 x 4096 bfloat16 errors behind a
// gelu: 41 and 36 us, 3.3 and 4.7 TB/s; the first is held up by its arithmetic
// (27 instructions a value, two of them quarter-rate) as much as by memory:
// neither four rows in flight nor twice the workgroups changed it.
#include "dfp8_convert.h"

namespace ionn {
namespace dfp8 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t block_max(uint32_t v) {
    __shared__ uint32_t red[kThreads / 64];
    v = wave_max_u32(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return max(max(red[0], red[1]), max(red[2], red[3]));
}

// ---- a floating tensor -------------------------------------------------------

template <class T>
__global__ __launch_bounds__(kThreads) void max_kernel(const T *__restrict__ x, int64_t n,
                                                       uint32_t *__restrict__ part) {
    constexpr int VE = 16 / sizeof(T);
    uint32_t m = 0;
    const int64_t step = int64_t(gridDim.x) * kThreads * VE;
    for (int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * VE; i < n; i += step) {
        const auto v = load_raw<T, VE>(x + i, int(n - i < VE ? n - i : VE));
#pragma unroll
        for (int e = 0; e < VE; ++e) m = max(m, mag_bits(float(v[e])));
    }
    m = block_max(m);
    if (threadIdx.x == 0) part[blockIdx.x] = m;
}

__device__ __forceinline__ void store_bytes(int8_t *p, const uint32_t *q, int count, int valid) {
    if (valid >= count) {
        if (count == 8)
            *reinterpret_cast<__attribute__((aligned(1))) uint64_t *>(p) =
                uint64_t(pack4_u8(q[0], q[1], q[2], q[3])) | uint64_t(pack4_u8(q[4], q[5], q[6], q[7])) << 32;
        else
            *reinterpret_cast<__attribute__((aligned(1))) uint32_t *>(p) = pack4_u8(q[0], q[1], q[2], q[3]);
        return;
    }
    for (int e = 0; e < valid; ++e) p[e] = int8_t(q[e]);
}

// The largest of the first pass's maxima.
__device__ __forceinline__ uint32_t all_max(const uint32_t *__restrict__ part, int nparts) {
    uint32_t m = 0;
    for (int i = threadIdx.x; i < nparts; i += kThreads) m = max(m, part[i]);
    return block_max(m);
}

// GIVEN: part is a producer's maximum, taken before it rounded its values to
// T; rounding keeps their order, so it is rounded here (and an infinity that
// only the type made shows).
template <class T, bool GIVEN>
__global__ __launch_bounds__(kThreads) void round_kernel(const T *__restrict__ x, int64_t n,
                                                         const uint32_t *__restrict__ part, int nparts,
                                                         int8_t *__restrict__ out, int32_t *__restrict__ e_out,
                                                         int32_t *__restrict__ status) {
    constexpr int VE = 16 / sizeof(T);
    const uint32_t m = GIVEN ? mag_bits(float(T(__uint_as_float(*part)))) : all_max(part, nparts);
    const int E = dfp8_exponent(m);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *e_out = E;
        if (status) *status = dfp8_status(m, E);
    }
    const int64_t step = int64_t(gridDim.x) * kThreads * VE;
    for (int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * VE; i < n; i += step) {
        const int valid = int(n - i < VE ? n - i : VE);
        const auto v = load_raw<T, VE>(x + i, valid);
        uint32_t q[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) q[e] = dfp8_mantissa(float(v[e]), -E);
        store_bytes(out + i, q, VE, valid);
    }
}

// ---- the error behind an activation ------------------------------------------

// Workgroup (strip, chunk): the strip's columns over the chunk's rows, four
// wavefronts of 64 / lanes rows each at a time.
template <class T, int ACT>
__global__ __launch_bounds__(kThreads) void act_sums_kernel(const T *__restrict__ dY, const T *__restrict__ Z,
                                                            int64_t B, int OUT, int lanes_log, int64_t chunk_rows,
                                                            uint32_t *__restrict__ part_max,
                                                            float *__restrict__ part_sum) {
    constexpr int VE = 16 / sizeof(T);
    __shared__ float fold[kThreads / 64][64 * VE];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lanes = 1 << lanes_log, per_wave = 64 >> lanes_log;
    const int c = (int(blockIdx.x) * lanes + (lane & (lanes - 1))) * VE;
    const int64_t r1 = min(B, int64_t(blockIdx.y + 1) * chunk_rows);
    float s[VE] = {};
    uint32_t m = 0;
    if (c < OUT) {
        const int valid = OUT - c;
        const int step = (kThreads / 64) * per_wave;
        auto add = [&](const typename Vec<T, VE>::type &y, const typename Vec<T, VE>::type &z) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float d = ACT == IONN_ACT_NONE ? float(y[e]) : float(y[e]) * act_grad<ACT, kTermsGrad>(float(z[e]));
                s[e] += d;
                m = max(m, mag_bits(d));  // (past a row's end dY, and so d, is 0)
            }
        };
        int64_t r = int64_t(blockIdx.y) * chunk_rows + wave * per_wave + (lane >> lanes_log);
        // four rows' loads in flight
        for (; r + 3 * step < r1; r += 4 * step) {
            typename Vec<T, VE>::type y[4], z[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                y[u] = load_raw<T, VE>(dY + (r + u * step) * OUT + c, valid);
                if (ACT != IONN_ACT_NONE) z[u] = load_raw<T, VE>(Z + (r + u * step) * OUT + c, valid);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) add(y[u], z[u]);
        }
        for (; r < r1; r += step) {
            const auto y = load_raw<T, VE>(dY + r * OUT + c, valid);
            typename Vec<T, VE>::type z = y;
            if (ACT != IONN_ACT_NONE) z = load_raw<T, VE>(Z + r * OUT + c, valid);
            add(y, z);
        }
    }
    // the row groups of a wavefront, then the wavefronts
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        for (int off = lanes; off < 64; off <<= 1) s[e] += __shfl_xor(s[e], off, 64);
        fold[wave][(lane & (lanes - 1)) * VE + e] = s[e];
    }
    m = block_max(m);  // (its barrier orders fold as well)
    if (threadIdx.x == 0) part_max[blockIdx.y * gridDim.x + blockIdx.x] = m;
    if (part_sum == nullptr) return;
    for (int i = threadIdx.x; i < lanes * VE; i += kThreads) {
        const int col = int(blockIdx.x) * lanes * VE + i;
        if (col < OUT)
            part_sum[int64_t(blockIdx.y) * OUT + col] = (fold[0][i] + fold[1][i]) + (fold[2][i] + fold[3][i]);
    }
}

// Workgroups below n_round round the errors; those from it on add up the
// chunks' column sums, 64 columns at a time, every fourth chunk per wavefront.
template <class T, int ACT>
__global__ __launch_bounds__(kThreads) void act_round_kernel(const T *__restrict__ dY, const T *__restrict__ Z,
                                                             int64_t n, int OUT, const uint32_t *__restrict__ part_max,
                                                             int nparts, int n_round, const float *__restrict__ part_sum,
                                                             int chunks, int8_t *__restrict__ dZ8,
                                                             int32_t *__restrict__ edZ, float *__restrict__ gb,
                                                             int32_t *__restrict__ status) {
    constexpr int VE = 16 / sizeof(T);
    if (int(blockIdx.x) >= n_round) {
        __shared__ float red[kThreads / 64][64];
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int64_t step = (int64_t(gridDim.x) - n_round) * 64;
        for (int64_t c0 = int64_t(int(blockIdx.x) - n_round) * 64; c0 < OUT; c0 += step) {
            const int64_t c = c0 + lane;
            float s = 0.0f;
            if (c < OUT) {
#pragma unroll 8
                for (int k = wave; k < chunks; k += kThreads / 64) s += part_sum[int64_t(k) * OUT + c];
            }
            red[wave][lane] = s;
            __syncthreads();
            if (wave == 0 && c < OUT) gb[c] = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
            __syncthreads();
        }
        return;
    }
    const uint32_t m = all_max(part_max, nparts);
    const int E = dfp8_exponent(m);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *edZ = E;
        if (status) *status = dfp8_status(m, E);
    }
    const int64_t step = int64_t(n_round) * kThreads * VE;
    auto put = [&](int64_t i, const typename Vec<T, VE>::type &y, const typename Vec<T, VE>::type &z,
                   int valid) __attribute__((always_inline)) {
        uint32_t q[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const float d = ACT == IONN_ACT_NONE ? float(y[e]) : float(y[e]) * act_grad<ACT, kTermsGrad>(float(z[e]));
            q[e] = dfp8_mantissa(d, -E);
        }
        store_bytes(dZ8 + i, q, VE, valid);
    };
    int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * VE;
    for (; i + step + VE <= n; i += 2 * step) {  // two pieces' loads in flight
        typename Vec<T, VE>::type y[2], z[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            y[u] = load_raw<T, VE>(dY + i + u * step);
            if (ACT != IONN_ACT_NONE) z[u] = load_raw<T, VE>(Z + i + u * step);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) put(i + u * step, y[u], z[u], VE);
    }
    for (; i < n; i += step) {
        const int valid = int(n - i < VE ? n - i : VE);
        const auto y = load_raw<T, VE>(dY + i, valid);
        typename Vec<T, VE>::type z = y;
        if (ACT != IONN_ACT_NONE) z = load_raw<T, VE>(Z + i, valid);
        put(i, y, z, valid);
    }
}

// Both passes in one workgroup, for an error of at most 16 values a thread:
// read once, no second launch.  Piece k of kOneValues / VE is strip k / groups
// of the columns, rows group k % groups: 16 wavefronts of 64 / lanes rows
// each.  One compute unit takes 3.9 us for 64 x 64 errors and 5.9 for 64 x 256
// (gelu, bfloat16) where the two launches take 7.7; past that it is the slower
// (11 us at 128 x 256).
constexpr int kOneThreads = 1024, kOneValues = 16;

template <class T, int ACT>
__global__ __launch_bounds__(kOneThreads) void act_one_kernel(const T *__restrict__ dY, const T *__restrict__ Z,
                                                              int B, int OUT, int lanes_log, int strips, int groups,
                                                              int8_t *__restrict__ dZ8, int32_t *__restrict__ edZ,
                                                              float *__restrict__ gb, int32_t *__restrict__ status) {
    constexpr int VE = 16 / sizeof(T), K = kOneValues / VE, kWaves = kOneThreads / 64;
    __shared__ float fold[kWaves][64 * VE];
    __shared__ uint32_t red[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lanes = 1 << lanes_log, per_wave = 64 >> lanes_log;
    const int row0 = wave * per_wave + (lane >> lanes_log), col0 = (lane & (lanes - 1)) * VE;
    const int pieces = strips * groups;
    const int64_t last = int64_t(B) * OUT - VE;  // >= 0: the caller checks
    float d[K][VE];
    uint32_t m = 0;
    // all loads in flight, none behind a lane's own condition: what lies past a
    // row's end is dropped below, and the tensor's last piece is read again
    // where its end cuts it
    typename Vec<T, VE>::type y[K], z[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (k < pieces) {
            const int c = (k / groups) * lanes * VE + col0, r = (k % groups) * kWaves * per_wave + row0;
            const int64_t at = min(int64_t(min(r, B - 1)) * OUT + c, last);
            y[k] = load_raw<T, VE>(dY + at);
            if (ACT != IONN_ACT_NONE) z[k] = load_raw<T, VE>(Z + at);
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (k < pieces) {
            const int c = (k / groups) * lanes * VE + col0, r = (k % groups) * kWaves * per_wave + row0;
            const int valid = r < B ? OUT - c : 0;
            const int64_t at = int64_t(r) * OUT + c;
            if (valid > 0 && at > last) {
                y[k] = load_raw<T, VE>(dY + at, valid);
                if (ACT != IONN_ACT_NONE) z[k] = load_raw<T, VE>(Z + at, valid);
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                d[k][e] = ACT == IONN_ACT_NONE ? float(y[k][e]) : float(y[k][e]) * act_grad<ACT, kTermsGrad>(float(z[k][e]));
                if (e >= valid) d[k][e] = 0.0f;
                m = max(m, mag_bits(d[k][e]));
            }
        }
    }
    m = wave_max_u32(m);
    if (lane == 0) red[wave] = m;
    __syncthreads();
    m = red[lane & (kWaves - 1)];
    m = wave_max_u32(m);
    const int E = dfp8_exponent(m);
    if (threadIdx.x == 0) {
        *edZ = E;
        if (status) *status = dfp8_status(m, E);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (k < pieces) {
            const int c = (k / groups) * lanes * VE + col0, r = (k % groups) * kWaves * per_wave + row0;
            uint32_t q[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) q[e] = dfp8_mantissa(d[k][e], -E);
            store_bytes(dZ8 + int64_t(r) * OUT + c, q, VE, r < B ? OUT - c : 0);
        }
    }
    if (gb == nullptr) return;
    // a strip's rows in a thread, then the row groups of a wavefront, then the wavefronts
    float s[VE] = {};
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (k < pieces) {
#pragma unroll
            for (int e = 0; e < VE; ++e) s[e] += d[k][e];
            if (k % groups == groups - 1) {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    for (int off = lanes; off < 64; off <<= 1) s[e] += __shfl_xor(s[e], off, 64);
                    fold[wave][col0 + e] = s[e];
                    s[e] = 0.0f;
                }
                __syncthreads();
                const int i = threadIdx.x, col = (k / groups) * lanes * VE + i;
                if (i < lanes * VE && col < OUT) {
                    float v = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) v += fold[w][i];
                    gb[col] = v;
                }
                __syncthreads();
            }
        }
    }
}

// Workgroups for a pass over n values of es bytes, 16 bytes per thread.
unsigned pass_groups(int64_t n, size_t es, int64_t most) {
    const int64_t per = kThreads * int64_t(16 / es);
    const int64_t b = (n + per - 1) / per;
    return unsigned(b < most ? b : most);
}

}  // namespace

ActLayout act_layout(int64_t B, int64_t OUT, size_t es) {
    const int64_t ve = int64_t(16 / es);
    ActLayout a;
    a.lanes = 1;
    while (a.lanes < 64 && a.lanes * ve < OUT) a.lanes *= 2;
    const int64_t strips = (OUT + a.lanes * ve - 1) / (a.lanes * ve);
    a.strips = int(strips);
    // at least four rows per lane in a range, and about kMaxParts workgroups
    const int64_t least = int64_t(4) * (kThreads / a.lanes);
    int64_t chunks = kMaxParts / strips;
    if (chunks > (B + least - 1) / least) chunks = (B + least - 1) / least;
    if (chunks < 1) chunks = 1;
    a.rows = (B + chunks - 1) / chunks;
    a.chunks = int((B + a.rows - 1) / a.rows);
    return a;
}

size_t act_workspace_bytes(int64_t B, int64_t OUT) {
    size_t most = 0;
    for (size_t es : {size_t(2), size_t(4)}) {
        const ActLayout a = act_layout(B, OUT, es);
        const size_t maxima = (size_t(a.strips) * a.chunks * sizeof(uint32_t) + 15) & ~size_t(15);
        const size_t b = maxima + size_t(a.chunks) * OUT * sizeof(float);
        most = b > most ? b : most;
    }
    return (most + 15) & ~size_t(15);
}

int launch_act_bwd(const void *dY, const void *Z, int act, int dtype, int64_t B, int64_t OUT, int8_t *dZ8,
                   int32_t *edZ, float *gb, int32_t *status, void *workspace, hipStream_t st) {
    const ActLayout a = act_layout(B, OUT, dtype_size(dtype));
    const int nparts = a.strips * a.chunks;
    uint32_t *maxima = static_cast<uint32_t *>(workspace);
    float *sums = gb ? reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                                 ((size_t(nparts) * sizeof(uint32_t) + 15) & ~size_t(15)))
                     : nullptr;
    int lanes_log = 0;
    while ((1 << lanes_log) < a.lanes) ++lanes_log;
    const int64_t groups = (B + 16 * (64 / a.lanes) - 1) / (16 * (64 / a.lanes));
    const bool one = a.strips * groups <= kOneValues / int64_t(16 / dtype_size(dtype)) &&
                     B * OUT >= int64_t(16 / dtype_size(dtype));
    const unsigned n_round = pass_groups(B * OUT, dtype_size(dtype), 2048);
    // (at most 2^20: one for each 64 of 2^30 columns and the others would be too many threads)
    const unsigned n_sum = gb ? unsigned(OUT <= int64_t(64) << 20 ? (OUT + 63) / 64 : int64_t(1) << 20) : 0u;
    with_dtype(dtype, [&](auto tag) {
        using T = decltype(tag);
        const T *y = static_cast<const T *>(dY), *z = static_cast<const T *>(Z);
        with_act(act, [&](auto ac) {
            constexpr int ACT = decltype(ac)::value;
            if (one) {
                act_one_kernel<T, ACT><<<dim3(1), dim3(kOneThreads), 0, st>>>(
                    y, z, int(B), int(OUT), lanes_log, a.strips, int(groups), dZ8, edZ, gb, status);
                return;
            }
            act_sums_kernel<T, ACT><<<dim3(unsigned(a.strips), unsigned(a.chunks)), dim3(kThreads), 0, st>>>(
                y, z, B, int(OUT), lanes_log, a.rows, maxima, sums);
            act_round_kernel<T, ACT><<<dim3(n_round + n_sum), dim3(kThreads), 0, st>>>(
                y, z, B * OUT, int(OUT), maxima, nparts, int(n_round), sums, a.chunks, dZ8, edZ, gb, status);
        });
    });
    return check_launch("dfp8_linear_bwd");
}

}  // namespace dfp8
}  // namespace ionn

using namespace ionn;
using namespace ionn::dfp8;

extern "C" {

size_t dfp8_from_float_workspace_bytes(void) { return kMaxParts * sizeof(uint32_t); }

int dfp8_from_float(const void *x, int dtype, int64_t n, const uint32_t *absmax, int8_t *out, int32_t *e_out,
                    int32_t *status_out, void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    IONN_REQUIRE(dtype_ok(dtype), IONN_ERR_ARG, "dfp8_from_float: dtype = %d", dtype);
    IONN_REQUIRE(n >= 1 && n <= (int64_t(1) << 40), IONN_ERR_SHAPE, "dfp8_from_float: n = %lld", (long long)n);
    IONN_REQUIRE(x && out && e_out, IONN_ERR_ARG, "dfp8_from_float: NULL argument");
    IONN_REQUIRE(aligned(x, dtype_size(dtype)) && aligned(e_out, 4) && aligned(status_out, 4) && aligned(absmax, 4),
                 IONN_ERR_ALIGN, "dfp8_from_float: x must be aligned to its element size, the scalars to 4 bytes");
    IONN_REQUIRE(absmax || (workspace && aligned(workspace, 4) && workspace_bytes >= dfp8_from_float_workspace_bytes()),
                 IONN_ERR_WORKSPACE, "dfp8_from_float: needs a 4-byte aligned workspace of %zu bytes",
                 dfp8_from_float_workspace_bytes());
    hipStream_t st = as_stream(stream);
    uint32_t *part = static_cast<uint32_t *>(workspace);
    int nparts = 0;
    with_dtype(dtype, [&](auto tag) {
        using T = decltype(tag);
        const T *p = static_cast<const T *>(x);
        if (!absmax) {
            nparts = int(pass_groups(n, sizeof(T), kMaxParts));
            max_kernel<T><<<dim3(unsigned(nparts)), dim3(kThreads), 0, st>>>(p, n, part);
        }
        const dim3 grid{pass_groups(n, sizeof(T), 2048)}, block{kThreads};
        if (absmax) round_kernel<T, true><<<grid, block, 0, st>>>(p, n, absmax, 1, out, e_out, status_out);
        else round_kernel<T, false><<<grid, block, 0, st>>>(p, n, part, nparts, out, e_out, status_out);
    });
    return check_launch("dfp8_from_float");
}

}  // extern "C"
