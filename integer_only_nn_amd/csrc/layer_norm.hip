// Layer norm over the rows of a floating tensor, and its gradient ("Mixed
// Precision Training of Convolutional Neural Networks using Integer
// Operations", section 4: the operations around the integer kernels run in
// floating point).
//
//   y = (x - mean) * rstd * gamma + beta
//   dx = rstd * (d - mean(d) - h * mean(d h)) + dres, h = (x - mean) rstd,
//   d = dy gamma;  dgamma = sum_rows dy h, dbeta = sum_rows dy
//
// Both directions are bound by HBM: x read and y written once (forward), x
// and dy read and dx written once (backward).  So a row is read into
// registers, where its sums are taken in two passes (the squares around the
// mean, which a one-pass form loses for a mean far from 0), and a thread keeps
// the columns it owns from row to row: gamma, beta and the column sums of the
// backward pass stay in its registers, and the sums leave as one partial row
// per workgroup, added in a second, fixed-order pass.  The next row's loads are
// in flight while a row is reduced (forward 40.6 us without, 8192 x 4096
// bf16).  Measured: forward 8192 x 4096 bf16 27 us (5.0 TB/s, a large copy
// reaches 5.2); backward 45 us and 5 for the second pass; 25088 x 256 float32
// backward 15.4 and 3.9 us; one row of 4096 forward 3.1 us.
#include "float_ops.h"

namespace ionn {
namespace {

constexpr int kMaxParts = 512;      // workgroups, and partial rows, of the backward pass
constexpr int kThreads = 256;

// Sum of v over the TPR threads that share a row (whole wavefronts); every
// one of them gets it.  buf: one float per wavefront, twice over, so that
// one barrier per sum suffices (ph alternates).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*buf)[TPR / 64 + 1], int &ph) {
    v = wave_sum(v);
    if (TPR == 64) return v;
    float *b = buf[ph];
    ph ^= 1;
    if ((threadIdx.x & 63) == 0) b[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = b[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) s += b[w];
    return s;
}

// Rows of up to TPR * NV * VE columns: thread t of the TPR threads of a row
// holds columns (i TPR + t) VE .. + VE - 1.
template <class T, int VE, int TPR, int NV>
__global__ __launch_bounds__(TPR < kThreads ? kThreads : TPR) void norm_fwd_kernel(
    const T *x, const float *__restrict__ gamma, const float *__restrict__ beta, float eps, T *y,
    float *__restrict__ mean_out, float *__restrict__ rstd_out, int64_t rows, int cols, float n_cols,
    uint32_t *absmax) {
    __shared__ float buf[2][TPR / 64 + 1];
    constexpr int kRows = TPR < kThreads ? kThreads / TPR : 1;  // rows a workgroup takes at once
    constexpr bool kHold = NV * VE <= 16;                       // gamma and beta stay in registers
    const int t = threadIdx.x % TPR;
    const int64_t step = int64_t(gridDim.x) * kRows;
    int64_t r = int64_t(blockIdx.x) * kRows + threadIdx.x / TPR;
    int ph = 0;
    uint32_t top = 0;
    // the next row's loads go out before this row's sums are taken
    typename Vec<T, VE>::type raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * VE;
        raw[i] = load_raw<T, VE>(x + r * cols + c, r < rows ? cols - c : 0);
    }
    typename Vec<float, VE>::type gh[kHold ? NV : 1], bh[kHold ? NV : 1];
    if (kHold) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VE;
            gh[i] = gamma ? load_raw<float, VE>(gamma + c, cols - c) : typename Vec<float, VE>::type(1.0f);
            bh[i] = load_raw<float, VE>(beta + c, beta ? cols - c : 0);
        }
    }
    for (; r < rows; r += step) {
        float v[NV][VE];
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                v[i][e] = float(raw[i][e]);
                s += v[i][e];
            }
        if (r + step < rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + t) * VE;
                raw[i] = load_raw<T, VE>(x + (r + step) * cols + c, cols - c);
            }
        }
        const float mean = row_sum<TPR>(s, buf, ph) / n_cols;
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float d = (i * TPR + t) * VE + e < cols ? v[i][e] - mean : 0.0f;
                v[i][e] = d;
                q += d * d;
            }
        const float rstd = 1.0f / sqrtf(row_sum<TPR>(q, buf, ph) / n_cols + eps);
        if (t == 0) {
            if (mean_out) mean_out[r] = mean;
            if (rstd_out) rstd_out[r] = rstd;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VE;
            const int valid = cols - c;
            if (valid <= 0) continue;
            typename Vec<float, VE>::type g, b;
            if (kHold) {
                g = gh[i];
                b = bh[i];
            } else {
                g = gamma ? load_raw<float, VE>(gamma + c, valid) : typename Vec<float, VE>::type(1.0f);
                b = load_raw<float, VE>(beta + c, beta ? valid : 0);
            }
            float o[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) o[e] = v[i][e] * rstd * g[e] + b[e];
            if (absmax) {
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (e < valid) top = max(top, mag_bits(o[e]));
            }
            store_vec<T, VE>(y + r * cols + c, o, valid);
        }
    }
    if (absmax) {
        top = wave_max_u32(top);
        if ((threadIdx.x & 63) == 0) publish_max_u32(absmax, top);
    }
}

// Rows of any length, one workgroup each, read once per sum.
template <class T, int VE>
__global__ __launch_bounds__(1024) void norm_fwd_long_kernel(const T *x, const float *__restrict__ gamma,
                                                             const float *__restrict__ beta, float eps, T *y,
                                                             float *__restrict__ mean_out,
                                                             float *__restrict__ rstd_out, int64_t rows, int cols,
                                                             float n_cols, uint32_t *absmax) {
    __shared__ float buf[2][17];
    int ph = 0;
    uint32_t top = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *xr = x + r * cols;
        float s = 0.0f;
        for (int64_t c = int64_t(threadIdx.x) * VE; c < cols; c += 1024 * VE) {
            const auto raw = load_raw<T, VE>(xr + c, int(cols - c));
#pragma unroll
            for (int e = 0; e < VE; ++e) s += float(raw[e]);
        }
        const float mean = row_sum<1024>(s, buf, ph) / n_cols;
        float q = 0.0f;
        for (int64_t c = int64_t(threadIdx.x) * VE; c < cols; c += 1024 * VE) {
            const auto raw = load_raw<T, VE>(xr + c, int(cols - c));
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float d = c + e < cols ? float(raw[e]) - mean : 0.0f;
                q += d * d;
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<1024>(q, buf, ph) / n_cols + eps);
        if (threadIdx.x == 0) {
            if (mean_out) mean_out[r] = mean;
            if (rstd_out) rstd_out[r] = rstd;
        }
        for (int64_t c = int64_t(threadIdx.x) * VE; c < cols; c += 1024 * VE) {
            const int valid = int(cols - c);
            const auto raw = load_raw<T, VE>(xr + c, valid);
            float o[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                o[e] = (float(raw[e]) - mean) * rstd;
                if (e < valid) {
                    if (gamma) o[e] *= gamma[c + e];
                    if (beta) o[e] += beta[c + e];
                    top = max(top, mag_bits(o[e]));
                }
            }
            store_vec<T, VE>(y + r * cols + c, o, valid);
        }
    }
    if (absmax) {
        top = wave_max_u32(top);
        if ((threadIdx.x & 63) == 0) publish_max_u32(absmax, top);
    }
}

// Threads of a workgroup of the backward pass: short rows, one wavefront
// each, go eight to a workgroup, so that few partial rows leave it.
constexpr int bwd_threads(int tpr) { return tpr == 64 ? 512 : tpr; }

// part: [gridDim.x][2][cols], the workgroups' sums of dy h and dy (NULL: not asked for).
template <class T, int VE, int TPR, int NV>
__global__ __launch_bounds__(bwd_threads(TPR)) void norm_bwd_kernel(
    const T *dy, const T *__restrict__ x, const float *__restrict__ mean, const float *__restrict__ rstd,
    const float *__restrict__ gamma, const T *dres, T *dx, float *__restrict__ part, int64_t rows, int cols,
    float n_cols) {
    constexpr int kRows = bwd_threads(TPR) / TPR;
    __shared__ float buf[2][TPR / 64 + 1];
    __shared__ float fold[kRows > 1 ? kRows * NV * VE * TPR : 1];
    const int t = threadIdx.x % TPR, rg = threadIdx.x / TPR;
    int ph = 0;
    float g[NV][VE], sg[NV][VE], sb[NV][VE];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * VE;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            g[i][e] = gamma && c + e < cols ? gamma[c + e] : 1.0f;
            sg[i][e] = sb[i][e] = 0.0f;
        }
    }
    // the next row's loads go out before this row's sums are taken
    const int64_t step = int64_t(gridDim.x) * kRows;
    int64_t r = int64_t(blockIdx.x) * kRows + rg;
    typename Vec<T, VE>::type rx[NV], ry[NV];
    float mu_next = 0.0f, rs_next = 0.0f;
    auto load_row = [&](int64_t row) __attribute__((always_inline)) {
        mu_next = mean[row];
        rs_next = rstd[row];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VE;
            rx[i] = load_raw<T, VE>(x + row * cols + c, cols - c);
            ry[i] = load_raw<T, VE>(dy + row * cols + c, cols - c);
        }
    };
    if (r < rows) load_row(r);
    for (; r < rows; r += step) {
        const float mu = mu_next, rs = rs_next;
        float h[NV][VE], d[NV][VE];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VE;
#pragma unroll
            for (int e = 0; e < VE; ++e) h[i][e] = (float(rx[i][e]) - mu) * rs;
            // past the row's end dy is 0, and so is every sum's term where h is
            // finite, which mu rs need not be
            if (cols - c < VE) {
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (c + e >= cols) h[i][e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float a = float(ry[i][e]);
                sg[i][e] += a * h[i][e];
                sb[i][e] += a;
                d[i][e] = a * g[i][e];
                s1 += d[i][e];
                s2 += d[i][e] * h[i][e];
            }
        }
        if (r + step < rows) load_row(r + step);
        const float c1 = row_sum<TPR>(s1, buf, ph) / n_cols;
        const float c2 = row_sum<TPR>(s2, buf, ph) / n_cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VE;
            const int valid = cols - c;
            if (valid <= 0) continue;
            float o[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) o[e] = rs * (d[i][e] - c1 - h[i][e] * c2);
            if (dres) {
                const auto rr = load_raw<T, VE>(dres + r * cols + c, valid);
#pragma unroll
                for (int e = 0; e < VE; ++e) o[e] += float(rr[e]);
            }
            store_vec<T, VE>(dx + r * cols + c, o, valid);
        }
    }
    if (part == nullptr) return;
    float *p = part + int64_t(blockIdx.x) * 2 * cols;
    // the workgroup's row groups one after the other, dy h and then dy
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float(&s)[NV][VE] = k ? sb : sg;
        if (kRows > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) fold[((rg * NV + i) * VE + e) * TPR + t] = s[i][e];
            __syncthreads();
            if (rg > 0) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    float v = s[i][e];
#pragma unroll
                    for (int o = 1; o < kRows; ++o) v += fold[((o * NV + i) * VE + e) * TPR + t];
                    s[i][e] = v;
                }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VE;
            if (c < cols) store_vec<float, VE>(p + int64_t(k) * cols + c, s[i], cols - c);
        }
    }
}

// Rows of any length: one workgroup each, both sums first and then dx.  dx
// may be dy: a workgroup reads a place before it writes it, and the column
// sums are taken by norm_bwd_cols_kernel before this kernel runs.
template <class T, int VE>
__global__ __launch_bounds__(1024) void norm_bwd_long_kernel(const T *dy, const T *__restrict__ x,
                                                             const float *__restrict__ mean,
                                                             const float *__restrict__ rstd,
                                                             const float *__restrict__ gamma, const T *dres, T *dx,
                                                             int64_t rows, int cols, float n_cols) {
    __shared__ float buf[2][17];
    int ph = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const float mu = mean[r], rs = rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = int64_t(threadIdx.x) * VE; c < cols; c += 1024 * VE) {
            const int valid = int(cols - c);
            const auto rx = load_raw<T, VE>(x + r * cols + c, valid);
            const auto ry = load_raw<T, VE>(dy + r * cols + c, valid);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float d = float(ry[e]) * (gamma && e < valid ? gamma[c + e] : 1.0f);
                s1 += d;
                s2 += d * (e < valid ? (float(rx[e]) - mu) * rs : 0.0f);
            }
        }
        const float c1 = row_sum<1024>(s1, buf, ph) / n_cols;
        const float c2 = row_sum<1024>(s2, buf, ph) / n_cols;
        for (int64_t c = int64_t(threadIdx.x) * VE; c < cols; c += 1024 * VE) {
            const int valid = int(cols - c);
            const auto rx = load_raw<T, VE>(x + r * cols + c, valid);
            const auto ry = load_raw<T, VE>(dy + r * cols + c, valid);
            float o[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float d = float(ry[e]) * (gamma && e < valid ? gamma[c + e] : 1.0f);
                o[e] = rs * (d - c1 - (float(rx[e]) - mu) * rs * c2);
                if (dres && e < valid) o[e] += float(dres[r * cols + c + e]);
            }
            store_vec<T, VE>(dx + r * cols + c, o, valid);
        }
    }
}

// Column sums for the rows that norm_bwd_long_kernel takes: thread = VE
// columns, blockIdx.y = a range of rows, the same layout of partial sums.
template <class T, int VE>
__global__ __launch_bounds__(kThreads) void norm_bwd_cols_kernel(const T *__restrict__ dy, const T *__restrict__ x,
                                                                 const float *__restrict__ mean,
                                                                 const float *__restrict__ rstd,
                                                                 float *__restrict__ part, int64_t rows, int cols) {
    const int64_t c = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * VE;
    if (c >= cols) return;
    const int valid = int(cols - c);
    float sg[VE] = {}, sb[VE] = {};
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const float mu = mean[r], rs = rstd[r];
        const auto rx = load_raw<T, VE>(x + r * cols + c, valid);
        const auto ry = load_raw<T, VE>(dy + r * cols + c, valid);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            sg[e] += float(ry[e]) * ((float(rx[e]) - mu) * rs);
            sb[e] += float(ry[e]);
        }
    }
    float *p = part + int64_t(blockIdx.y) * 2 * cols + c;
    store_vec<float, VE>(p, sg, valid);
    store_vec<float, VE>(p + cols, sb, valid);
}

// The partial rows added up: 64 columns (of the 2 * cols) at a time per
// workgroup, each by 16 threads that take every 16th partial row, then those 16
// in order.
constexpr int kSumGroups = 16;
constexpr int64_t kSumBlocks = 65536;  // at most (one for each 64 of 2^28 sums would be too many threads to launch)
__global__ __launch_bounds__(64 * kSumGroups) void norm_sum_kernel(const float *__restrict__ part, int nparts,
                                                                   int64_t cols, float *__restrict__ dgamma,
                                                                   float *__restrict__ dbeta) {
    __shared__ float red[kSumGroups][64];
    const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
    for (int64_t c0 = int64_t(blockIdx.x) * 64; c0 < 2 * cols; c0 += int64_t(gridDim.x) * 64) {
        const int64_t c = c0 + lane;
        float s = 0.0f;
        if (c < 2 * cols) {
#pragma unroll 16
            for (int p = grp; p < nparts; p += kSumGroups) s += part[int64_t(p) * 2 * cols + c];
        }
        red[grp][lane] = s;
        __syncthreads();
        if (grp == 0 && c < 2 * cols) {
#pragma unroll
            for (int k = 1; k < kSumGroups; ++k) s += red[k][lane];
            float *out = c < cols ? dgamma : dbeta;
            if (out) out[c < cols ? c : c - cols] = s;
        }
        __syncthreads();
    }
}

// f(threads per row, vectors per thread) for a row of cols columns that fits
// in registers: one wavefront per row while that takes few vectors a lane (no
// barrier), then a workgroup of 256, then of 1024; false for longer rows.
// The backward pass holds five values per column where the forward holds
// one, so it takes more threads and fewer vectors.
template <int VE, bool BWD, class F>
bool with_shape(int64_t cols, F &&f) {
    const int64_t v = (cols + VE - 1) / VE;
    if (v <= 64) return f(IntC<64>{}, IntC<1>{}), true;
    if (v <= 128) return f(IntC<64>{}, IntC<2>{}), true;
    if (v <= 256) return f(IntC<256>{}, IntC<1>{}), true;
    if (v <= 512) return f(IntC<256>{}, IntC<2>{}), true;
    if constexpr (BWD) {
        if (v <= 1024) return f(IntC<1024>{}, IntC<1>{}), true;
    } else {
        if (v <= 1024) return f(IntC<256>{}, IntC<4>{}), true;
        if (v <= 4096) return f(IntC<1024>{}, IntC<4>{}), true;
    }
    return false;
}

// Workgroups of the backward pass, and partial rows: two of 256 threads per
// compute unit or one of more.  More keep more loads in flight, but leave more
// partial rows and deal the rows out less evenly: at 8192 x 4096 (bf16) two
// per unit took 44 us, one 53, three 50 and four 53; at 8192 x 1024 one of
// 512 threads took as long as two of 256 with half the partial rows.
int64_t bwd_groups(int64_t rows, int rows_per_group, int threads) {
    const int64_t b = (rows + rows_per_group - 1) / rows_per_group;
    int64_t most = int64_t(device_cus()) * (threads == 256 ? 2 : 1);
    if (most > kMaxParts) most = kMaxParts;
    return b < most ? b : most;
}

bool overlaps(const void *a, const void *b, size_t bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x != y && x < y + bytes && y < x + bytes;
}

}  // namespace
}  // namespace ionn

using namespace ionn;

extern "C" {

int ionn_layer_norm_fwd(const void *x, const float *gamma, const float *beta, double eps, void *y, float *mean,
                        float *rstd, int dtype, int64_t rows, int64_t cols, uint32_t *absmax_y, void *stream) {
    clear_error();
    IONN_REQUIRE(dtype_ok(dtype), IONN_ERR_ARG, "ionn_layer_norm_fwd: dtype = %d", dtype);
    IONN_REQUIRE(rows >= 0 && cols >= 0 && rows <= kMaxDim && cols <= kMaxDim, IONN_ERR_SHAPE,
                 "ionn_layer_norm_fwd: rows = %lld, cols = %lld", (long long)rows, (long long)cols);
    IONN_REQUIRE(eps >= 0.0 && eps <= 3.0e38, IONN_ERR_RANGE, "ionn_layer_norm_fwd: eps = %g", eps);
    if (rows == 0 || cols == 0) return IONN_OK;
    IONN_REQUIRE(x && y, IONN_ERR_ARG, "ionn_layer_norm_fwd: NULL tensor");
    const size_t es = dtype_size(dtype);
    IONN_REQUIRE(aligned(x, es) && aligned(y, es) && aligned(gamma, 4) && aligned(beta, 4) && aligned(mean, 4) &&
                     aligned(rstd, 4) && aligned(absmax_y, 4),
                 IONN_ERR_ALIGN, "ionn_layer_norm_fwd: tensors must be aligned to their element size");
    IONN_REQUIRE(!overlaps(x, y, size_t(rows) * cols * es), IONN_ERR_ARG,
                 "ionn_layer_norm_fwd: y may be x, but not overlap it otherwise");
    hipStream_t st = as_stream(stream);
    const float n = float(cols);
    with_dtype(dtype, [&](auto tag) {
        using T = decltype(tag);
        constexpr int VE = 16 / sizeof(T);
        const bool done = with_shape<VE, false>(cols, [&](auto tpr, auto nv) {
            constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
            constexpr int kRows = TPR < kThreads ? kThreads / TPR : 1;
            constexpr int kBlock = TPR < kThreads ? kThreads : TPR;
            // as many workgroups as are resident at once: rows are dealt out evenly
            int64_t blocks = (rows + kRows - 1) / kRows;
            const int64_t most = int64_t(device_cus()) * ((NV * VE > 8 ? 1024 : 2048) / kBlock);
            if (blocks > most) blocks = most;
            norm_fwd_kernel<T, VE, TPR, NV><<<dim3(unsigned(blocks)), dim3(kBlock), 0, st>>>(
                static_cast<const T *>(x), gamma, beta, float(eps), static_cast<T *>(y), mean, rstd, rows, int(cols), n,
                absmax_y);
        });
        if (!done) {
            const int64_t most = int64_t(device_cus()) * 2;
            norm_fwd_long_kernel<T, VE><<<dim3(unsigned(rows < most ? rows : most)), dim3(1024), 0, st>>>(
                static_cast<const T *>(x), gamma, beta, float(eps), static_cast<T *>(y), mean, rstd, rows, int(cols), n,
                absmax_y);
        }
    });
    return check_launch("ionn_layer_norm_fwd");
}

size_t ionn_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return 0;
    return size_t(rows < kMaxParts ? rows : kMaxParts) * 2 * size_t(cols) * sizeof(float);
}

int ionn_layer_norm_bwd(const void *dy, const void *x, const float *mean, const float *rstd, const float *gamma,
                        const void *dres, void *dx, float *dgamma, float *dbeta, int dtype, int64_t rows,
                        int64_t cols, void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    IONN_REQUIRE(dtype_ok(dtype), IONN_ERR_ARG, "ionn_layer_norm_bwd: dtype = %d", dtype);
    IONN_REQUIRE(rows >= 0 && cols >= 0 && rows <= kMaxDim && cols <= kMaxDim, IONN_ERR_SHAPE,
                 "ionn_layer_norm_bwd: rows = %lld, cols = %lld", (long long)rows, (long long)cols);
    if (cols == 0) return IONN_OK;
    const bool sums = dgamma || dbeta;
    IONN_REQUIRE(rows == 0 || (dy && x && mean && rstd && dx), IONN_ERR_ARG, "ionn_layer_norm_bwd: NULL tensor");
    const size_t es = dtype_size(dtype), bytes = size_t(rows) * cols * es;
    IONN_REQUIRE(aligned(dy, es) && aligned(x, es) && aligned(dx, es) && aligned(dres, es) && aligned(mean, 4) &&
                     aligned(rstd, 4) && aligned(gamma, 4) && aligned(dgamma, 4) && aligned(dbeta, 4),
                 IONN_ERR_ALIGN, "ionn_layer_norm_bwd: tensors must be aligned to their element size");
    IONN_REQUIRE(rows == 0 || (dx != x && !overlaps(dx, x, bytes) && !overlaps(dx, dy, bytes) &&
                               !overlaps(dx, dres, bytes)),
                 IONN_ERR_ARG, "ionn_layer_norm_bwd: dx may be dy or dres, but not overlap x or either in part");
    const size_t need = ionn_layer_norm_bwd_workspace_bytes(rows, cols);
    IONN_REQUIRE(!sums || need == 0 || (workspace && aligned(workspace, 16) && workspace_bytes >= need),
                 IONN_ERR_WORKSPACE, "ionn_layer_norm_bwd: needs a 16-byte aligned workspace of %zu bytes", need);
    hipStream_t st = as_stream(stream);
    float *part = sums ? static_cast<float *>(workspace) : nullptr;
    const float n = float(cols);
    int64_t groups = 0;
    if (rows > 0) {
        with_dtype(dtype, [&](auto tag) {
            using T = decltype(tag);
            constexpr int VE = 16 / sizeof(T);
            const T *tdy = static_cast<const T *>(dy), *tx = static_cast<const T *>(x);
            const T *tdr = static_cast<const T *>(dres);
            T *tdx = static_cast<T *>(dx);
            const bool done = with_shape<VE, true>(cols, [&](auto tpr, auto nv) {
                constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
                constexpr int kBlock = bwd_threads(TPR), kRows = kBlock / TPR;
                groups = bwd_groups(rows, kRows, kBlock);
                norm_bwd_kernel<T, VE, TPR, NV><<<dim3(unsigned(groups)), dim3(kBlock), 0, st>>>(
                    tdy, tx, mean, rstd, gamma, tdr, tdx, part, rows, int(cols), n);
            });
            if (!done) {
                if (sums) {
                    groups = bwd_groups(rows, 1, kThreads);
                    const dim3 grid(unsigned((cols + kThreads * VE - 1) / (kThreads * VE)), unsigned(groups));
                    norm_bwd_cols_kernel<T, VE><<<grid, dim3(kThreads), 0, st>>>(tdy, tx, mean, rstd, part, rows,
                                                                                 int(cols));
                }
                const int64_t most = int64_t(device_cus()) * 2;
                norm_bwd_long_kernel<T, VE><<<dim3(unsigned(rows < most ? rows : most)), dim3(1024), 0, st>>>(
                    tdy, tx, mean, rstd, gamma, tdr, tdx, rows, int(cols), n);
            }
        });
        if (int rc = check_launch("ionn_layer_norm_bwd")) return rc;
    }
    if (sums) {
        const int64_t blocks = (2 * cols + 63) / 64;
        norm_sum_kernel<<<dim3(unsigned(blocks < kSumBlocks ? blocks : kSumBlocks)), dim3(64 * kSumGroups), 0, st>>>(
            part, int(groups), cols, dgamma, dbeta);
        return check_launch("ionn_layer_norm_bwd");
    }
    return IONN_OK;
}

}  // extern "C"
