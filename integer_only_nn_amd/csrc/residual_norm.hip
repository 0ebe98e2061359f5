// What lies between two blocks of a residual stream, in one pass: the norm after
// a block, its gate, the scaled residual and the norm before the next block; and
// the gradient of it all ("Mixed Precision Training of Convolutional Neural
// Networks using Integer Operations", section 4: the operations around the
// integer kernels run in floating point).
//
//   p = N_a(a),  y = alpha x + gate p,  n = N_y(y)
//   t = dy + N_y'(dn),  dx = alpha t,  da = N_a'(gate t),
//   dgate = sum t p,  dgamma_a = sum gate t h_a,  dbeta_a = sum gate t,
//   dgamma_y = sum dn h_y,  dbeta_y = sum dn
//
// with N a layer norm, an RMS norm or nothing, h the normalised row, and a gate
// of each `gate_rows` rows.  As single operations they would move the stream
// through memory once each; together a and x are read and y and n written once
// (forward), a, y, dy and dn read and da and dx written once (backward), and HBM
// bounds both.  A row lies in registers, up to eight columns a thread (sixteen in
// rows above 8192, where the forward pass reads its vectors again for every row, and
// in the backward pass of 16-bit rows of 513 to 1024), and the next row's loads are in
// flight while a row's sums are taken.  Measured, inputs out of the caches: forward 8192 x 4096 bf16 56 us (4.8 TB/s, a large copy reaches 5.2; 49
// where some of them are in); backward 84 us in the first pass (4.8 TB/s) and 8 in the
// second; 25088 x 256 float32 with 128 gates 32 and 9.
//
// The backward pass needs only four column sums for its five vectors: S1 = sum t
// and Sh = sum t h_a of the rows that share a gate give that gate's gradient
// (gamma_a Sh + beta_a S1) and, times the gate, dgamma_a and dbeta_a.  A
// workgroup takes a run of rows that share a gate and leaves one partial row of
// each, added in a second, fixed-order pass; where there are more gates than
// workgroups it takes whole gates, whose gradients it writes itself.
#include "float_ops.h"

namespace ionn {
namespace {

constexpr int64_t kMaxCols = 16384;
constexpr int kMaxGroups = 512;  // workgroups of the backward pass

// store_vec, past the caches where `stream`: tensors larger than an XCD's L2.  2048
// x 2048 bf16 forward 12.5 against 13.8 us, 8192 x 4096 49.4 against 55.2, backward
// 90.5 and 92.2, 25088 x 256 float32 backward 37.5 and 39.5; smaller ones take as
// long either way (1024 x 1024 8.8 and 13.8 us) and stay where the next kernel finds
// them.  With the kernel that reads them next (n to DFP-8; da's conversion in the
// Linear layer's backward pass) much of the lead goes: 2048 x 2048 16.6 and 17.9,
// backward 30.2 and 29.8, 25088 x 256 29.7 and 29.0, 53.8 and 52.9, and the largest,
// which the last-level cache would have held, are behind: 8192 x 4096 75.0 and 71.6,
// 125.4 and 120.8.
constexpr size_t kStreamBytes = size_t(4) << 20;
template <class T, int VE>
__device__ __forceinline__ void put_vec(T *p, const float (&x)[VE], int valid, bool stream) {
    if (!stream || valid < VE) return store_vec<T, VE>(p, x, valid);
    typename Vec<T, VE>::type v;
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = T(x[i]);
    __builtin_nontemporal_store(v, reinterpret_cast<typename Vec<T, VE>::loose *>(p));
}

template <int CTRL>
__device__ __forceinline__ float moved(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// The sum over an aligned group of N lanes, in each of them.
template <int N>
__device__ __forceinline__ float group_sum(float v) {
    v += moved<0xb1>(v);   // lane ^ 1
    v += moved<0x4e>(v);   // lane ^ 2
    v += moved<0x141>(v);  // the other four of eight
    if (N >= 16) v += moved<0x140>(v);  // the other eight of sixteen
    if (N >= 32) v += __shfl_xor(v, 16, 64);
    if (N >= 64) v += __shfl_xor(v, 32, 64);
    return v;
}

// Sums of v over the TPR threads that share a row (a part of a wavefront, or whole
// ones); every one of them gets them.  buf: the wavefronts' sums, twice over, so that one barrier
// per call suffices (ph alternates).
template <int TPR, int V>
__device__ __forceinline__ void row_sums(float (&v)[V], float (*buf)[V][TPR / 64 + 1], int &ph) {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = group_sum<(TPR < 64 ? TPR : 64)>(v[k]);
    if (TPR <= 64) return;
    float(*b)[TPR / 64 + 1] = buf[ph];
    ph ^= 1;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int k = 0; k < V; ++k) b[k][threadIdx.x >> 6] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < V; ++k) {
        v[k] = b[k][0];
#pragma unroll
        for (int w = 1; w < TPR / 64; ++w) v[k] += b[k][w];
    }
}

struct Norm {
    int kind;  // IONN_NORM_*
    const float *gamma, *beta;
    float *mean, *rstd;
};

struct Forward {
    const void *a, *x;
    void *y, *n;
    Norm na, ny;
    const float *gate;
    int64_t rows;
    uint32_t gate_rows;
    int cols;
    float alpha, eps;
    uint32_t *absmax;
    bool stream;
};

// The columns of a thread: (i TPR + t) VE .. + VE - 1, i < NV.
template <int VE, int TPR, int NV>
struct Cols {
    float v[NV][VE];
    // a float vector, or `none` without one; zeros past the end
    __device__ __forceinline__ void load(const float *p, int cols, int t, float none) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VE;
            const auto r = load_raw<float, VE>(p + c, p ? cols - c : 0);
#pragma unroll
            for (int e = 0; e < VE; ++e) v[i][e] = p || c + e >= cols ? r[e] : none;
        }
    }
};

// v := the normalised row (zeros past its end); returns mean and rstd.
template <int VE, int TPR, int NV>
__device__ __forceinline__ void normalise(float (&v)[NV][VE], int kind, float eps, int cols, int t,
                                          float (*buf)[1][TPR / 64 + 1], int &ph, float &mean, float &rstd) {
    const float n = float(cols);
    mean = 0.0f;
    if (kind == IONN_NORM_LAYER) {
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e) s[0] += v[i][e];
        row_sums<TPR, 1>(s, buf, ph);
        mean = s[0] / n;
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const float d = (i * TPR + t) * VE + e < cols ? v[i][e] - mean : 0.0f;
            v[i][e] = d;
            q[0] += d * d;
        }
    row_sums<TPR, 1>(q, buf, ph);
    rstd = 1.0f / sqrtf(q[0] / n + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) v[i][e] *= rstd;
}

constexpr int fwd_threads(int tpr) { return tpr <= 64 ? 256 : tpr; }

// The row of this thread among a workgroup's (scalar where a wavefront has one row, so
// that addresses are but for the column).
template <int TPR>
__device__ __forceinline__ int row_group() {
    const int g = int(threadIdx.x) / TPR;
    return TPR < 64 ? g : __builtin_amdgcn_readfirstlane(g);
}

template <class T, int VE, int TPR, int NV>
__global__ __launch_bounds__(fwd_threads(TPR)) void residual_norm_fwd_kernel(Forward f) {
    __shared__ float buf[2][1][TPR / 64 + 1];
    constexpr int kRows = fwd_threads(TPR) / TPR;  // rows a workgroup takes at once
    constexpr bool kHold = NV * VE <= 8;           // the vectors stay in registers
    typedef Cols<VE, TPR, NV> Vector;
    const T *a = static_cast<const T *>(f.a), *x = static_cast<const T *>(f.x);
    T *y = static_cast<T *>(f.y), *n = static_cast<T *>(f.n);
    const int t = threadIdx.x % TPR, cols = f.cols;
    const int64_t step = int64_t(gridDim.x) * kRows;
    int64_t r = int64_t(blockIdx.x) * kRows + row_group<TPR>();
    int ph = 0;
    uint32_t top = 0;
    typename Vec<T, VE>::type ra[NV], rx[NV];
    const auto load_row = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VE, valid = row < f.rows ? cols - c : 0;
            if (a) ra[i] = load_raw<T, VE>(a + row * cols + c, valid);
            rx[i] = load_raw<T, VE>(x + row * cols + c, valid);
        }
    };
    load_row(r);
    Vector ga, ba, gy, by, gate;
    const auto load_norms = [&]() __attribute__((always_inline)) {
        ga.load(f.na.gamma, cols, t, 1.0f);
        ba.load(f.na.beta, cols, t, 0.0f);
        gy.load(f.ny.gamma, cols, t, 1.0f);
        by.load(f.ny.beta, cols, t, 0.0f);
    };
    if (kHold) load_norms();
    uint32_t group = ~0u;
    for (; r < f.rows; r += step) {
        float v[NV][VE], w[NV][VE];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                v[i][e] = a ? float(ra[i][e]) : 0.0f;
                w[i][e] = f.alpha * float(rx[i][e]);
            }
        if (r + step < f.rows) load_row(r + step);
        if (!kHold) load_norms();
        const uint32_t g = f.gate ? uint32_t(r) / f.gate_rows : 0u;
        if (!kHold || g != group) gate.load(f.gate ? f.gate + int64_t(g) * cols : nullptr, cols, t, 1.0f);
        group = g;
        if (a) {
            if (f.na.kind != IONN_NORM_NONE) {
                float mean, rstd;
                normalise<VE, TPR, NV>(v, f.na.kind, f.eps, cols, t, buf, ph, mean, rstd);
                if (t == 0) {
                    if (f.na.mean) f.na.mean[r] = mean;
                    if (f.na.rstd) f.na.rstd[r] = rstd;
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) w[i][e] += gate.v[i][e] * (v[i][e] * ga.v[i][e] + ba.v[i][e]);
        }
        if (y) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + t) * VE;
                if (c < cols) put_vec<T, VE>(y + r * cols + c, w[i], cols - c, f.stream);
            }
        }
        if (n == nullptr) continue;
        float mean, rstd;
        normalise<VE, TPR, NV>(w, f.ny.kind, f.eps, cols, t, buf, ph, mean, rstd);
        if (t == 0) {
            if (f.ny.mean) f.ny.mean[r] = mean;
            if (f.ny.rstd) f.ny.rstd[r] = rstd;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VE, valid = cols - c;
            if (valid <= 0) continue;
            float o[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                o[e] = w[i][e] * gy.v[i][e] + by.v[i][e];
                if (e < valid) top = max(top, mag_bits(o[e]));
            }
            put_vec<T, VE>(n + r * cols + c, o, valid, f.stream);
        }
    }
    if (f.absmax) {
        top = wave_max_u32(top);
        if ((threadIdx.x & 63) == 0) publish_max_u32(f.absmax, top);
    }
}

// ---- backward ------------------------------------------------------------------

struct Backward {
    const void *dy, *dn, *a, *y;
    void *da, *dx;
    Norm na, ny;
    const float *gate;
    int64_t rows;
    uint32_t gate_rows, chunks;  // rows that share a gate; runs that they are cut into
    uint32_t chunk_rows, units;  // rows of a run; runs of all gates
    int cols;
    float alpha;
    // (kSums of two rows each are written)
    // [units][2][cols] (Sh, S1; with whole gates [workgroups][2][cols], dgamma_a
    // and dbeta_a), [workgroups][2][cols] (dgamma_y, dbeta_y); nullable
    float *part_a, *part_y;
    float *dgate;  // with whole gates; nullable
    bool stream;
};

constexpr int bwd_threads(int tpr) { return tpr <= 64 ? 512 : tpr; }

// h := the normalised rows of v (zeros past the end).
template <class T, int VE, int TPR, int NV>
__device__ __forceinline__ void rows_of(const typename Vec<T, VE>::type (&raw)[NV], float mean, float rstd, int cols,
                                        int t, float (&h)[NV][VE]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * VE;
#pragma unroll
        for (int e = 0; e < VE; ++e) h[i][e] = c + e < cols ? (float(raw[i][e]) - mean) * rstd : 0.0f;
    }
}

// d := rstd (d - mean(d) - h mean(d h)), the first mean for a layer norm only.
template <int VE, int TPR, int NV, bool SHIFT>
__device__ __forceinline__ void project(float (&d)[NV][VE], const float (&h)[NV][VE], int kind, float rstd, float n,
                                        float (*buf)[SHIFT ? 2 : 1][TPR / 64 + 1], int &ph) {
    constexpr int kLast = SHIFT ? 1 : 0;
    float s[SHIFT ? 2 : 1] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            if (SHIFT) s[0] += d[i][e];
            s[kLast] += d[i][e] * h[i][e];
        }
    row_sums<TPR, SHIFT ? 2 : 1>(s, buf, ph);
    const float c1 = SHIFT && kind == IONN_NORM_LAYER ? s[0] / n : 0.0f, c2 = s[kLast] / n;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) d[i][e] = rstd * (d[i][e] - c1 - h[i][e] * c2);
}

// WHOLE: a unit is a gate's rows, taken by one of a workgroup's row groups.  SHIFT:
// one of the norms is a layer norm, so that the sums S1 and dbeta_y are needed
// (without their registers two workgroups of 512 threads share a compute unit;
// two vectors a thread do not fit that many registers: 8192 x 4096 float32, layer
// norms, 173 us, and 280 where they are made to).
template <class T, int VE, int TPR, int NV, bool WHOLE, bool SHIFT>
__global__ __launch_bounds__(bwd_threads(TPR), NV == 1 && !(WHOLE && SHIFT) ? 4 : 1) void residual_norm_bwd_kernel(Backward b) {
    constexpr int kRows = bwd_threads(TPR) / TPR;
    typedef Cols<VE, TPR, NV> Vector;
    __shared__ float buf[2][SHIFT ? 2 : 1][TPR / 64 + 1];
    constexpr int kFolds = TPR < 64 ? bwd_threads(TPR) / 64 : kRows;  // rows of sums that a workgroup folds
    __shared__ float fold[kFolds > 1 ? kFolds * NV * VE * TPR : 1];
    const T *dy = static_cast<const T *>(b.dy), *dn = static_cast<const T *>(b.dn);
    const T *a = static_cast<const T *>(b.a), *y = static_cast<const T *>(b.y);
    T *da = static_cast<T *>(b.da), *dx = static_cast<T *>(b.dx);
    const int t = threadIdx.x % TPR, rg = row_group<TPR>(), cols = b.cols;
    const float n = float(cols);
    int ph = 0;
    // S: Sh, S1 of the run at hand; Y: dgamma_y, dbeta_y of all runs; A (WHOLE): dgamma_a, dbeta_a of all runs
    constexpr int kSums = SHIFT ? 2 : 1;
    Vector gy, ga, S[kSums], Y[kSums], A[WHOLE ? kSums : 1];
    gy.load(b.ny.gamma, cols, t, 1.0f);
#pragma unroll
    for (int k = 0; k < kSums; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e) Y[k].v[i][e] = A[WHOLE ? k : 0].v[i][e] = 0.0f;

    // the row groups of a workgroup (those of a wavefront first) one after the other, to two rows of partial sums
    const auto leave = [&](Vector *s, float *to) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < kSums; ++k) {
            if (kFolds > 1) {
                const int at = TPR < 64 ? int(threadIdx.x) >> 6 : rg;
#pragma unroll
                for (int off = TPR; off < 64; off <<= 1)
#pragma unroll
                    for (int i = 0; i < NV; ++i)
#pragma unroll
                        for (int e = 0; e < VE; ++e) s[k].v[i][e] += __shfl_xor(s[k].v[i][e], off, 64);
                __syncthreads();
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        if (TPR >= 64 || (threadIdx.x & 63) < TPR) fold[((at * NV + i) * VE + e) * TPR + t] = s[k].v[i][e];
                __syncthreads();
            }
            if (rg > 0) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + t) * VE;
                float o[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    o[e] = s[k].v[i][e];
#pragma unroll
                    for (int g = 1; g < kFolds; ++g) o[e] += fold[((g * NV + i) * VE + e) * TPR + t];
                }
                if (c < cols) store_vec<float, VE>(to + int64_t(k) * cols + c, o, cols - c);
            }
        }
    };

    typename Vec<T, VE>::type r_dy[NV], r_dn[NV], r_a[NV], r_y[NV];
    float mean_a = 0.0f, rstd_a = 1.0f, mean_y = 0.0f, rstd_y = 1.0f;
    const auto load_row = [&](int64_t row) __attribute__((always_inline)) {
        if (b.na.rstd) rstd_a = b.na.rstd[row];
        if (b.na.mean) mean_a = b.na.mean[row];
        if (b.ny.rstd) rstd_y = b.ny.rstd[row];
        if (b.ny.mean) mean_y = b.ny.mean[row];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VE;
            if (dy) r_dy[i] = load_raw<T, VE>(dy + row * cols + c, cols - c);
            if (dn) r_dn[i] = load_raw<T, VE>(dn + row * cols + c, cols - c);
            if (dn) r_y[i] = load_raw<T, VE>(y + row * cols + c, cols - c);
            if (a) r_a[i] = load_raw<T, VE>(a + row * cols + c, cols - c);
        }
    };
    constexpr uint32_t kEach = WHOLE ? kRows : 1;  // units of a workgroup at once
    constexpr int kStep = WHOLE ? 1 : kRows;
    for (uint32_t unit = blockIdx.x * kEach + (WHOLE ? rg : 0); unit < b.units; unit += gridDim.x * kEach) {
        const uint32_t group = unit / b.chunks, chunk = unit - group * b.chunks;
        const int64_t first = int64_t(group) * b.gate_rows;
        const int64_t last = min(b.rows, first + min(int64_t(b.gate_rows), int64_t(chunk + 1) * b.chunk_rows));
        int64_t r = first + int64_t(chunk) * b.chunk_rows + (WHOLE ? 0 : rg);
        // gate and gamma_a as one factor
        {
            Vector g;
            g.load(b.gate ? b.gate + int64_t(group) * cols : nullptr, cols, t, 1.0f);
            ga.load(b.na.gamma, cols, t, 1.0f);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    ga.v[i][e] *= g.v[i][e];
#pragma unroll
                    for (int k = 0; k < kSums; ++k) S[k].v[i][e] = 0.0f;
                }
        }
        if (r < last) load_row(r);
        for (; r < last; r += kStep) {
            float d[NV][VE], h[NV][VE], past[NV][VE];
            const float mu_a = mean_a, rs_a = rstd_a, rs_y = rstd_y;
            if (dn) {
                rows_of<T, VE, TPR, NV>(r_y, SHIFT ? mean_y : 0.0f, rs_y, cols, t, h);
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float v = float(r_dn[i][e]);
                        Y[0].v[i][e] += v * h[i][e];
                        if (SHIFT) Y[kSums - 1].v[i][e] += v;
                        d[i][e] = v * gy.v[i][e];
                    }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) past[i][e] = dy ? float(r_dy[i][e]) : 0.0f;
            typename Vec<T, VE>::type row_a[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) row_a[i] = r_a[i];
            if (r + kStep < last) load_row(r + kStep);
            if (dn) {
                project<VE, TPR, NV, SHIFT>(d, h, b.ny.kind, rs_y, n, buf, ph);
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < VE; ++e) past[i][e] += d[i][e];
            }
            if (dx) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (i * TPR + t) * VE;
                    float o[VE];
#pragma unroll
                    for (int e = 0; e < VE; ++e) o[e] = b.alpha * past[i][e];
                    if (c < cols) put_vec<T, VE>(dx + r * cols + c, o, cols - c, b.stream);
                }
            }
            if (!a) continue;
            rows_of<T, VE, TPR, NV>(row_a, SHIFT ? mu_a : 0.0f, rs_a, cols, t, h);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    S[0].v[i][e] += past[i][e] * h[i][e];
                    if (SHIFT) S[kSums - 1].v[i][e] += past[i][e];
                    d[i][e] = past[i][e] * ga.v[i][e];
                }
            if (da) {
                if (b.na.kind != IONN_NORM_NONE) project<VE, TPR, NV, SHIFT>(d, h, b.na.kind, rs_a, n, buf, ph);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (i * TPR + t) * VE;
                    if (c < cols) put_vec<T, VE>(da + r * cols + c, d[i], cols - c, b.stream);
                }
            }
        }
        if (!WHOLE) {
            if (b.part_a) leave(S, b.part_a + int64_t(unit) * 2 * cols);
            continue;
        }
        Vector g, gamma, beta;
        g.load(b.gate + int64_t(group) * cols, cols, t, 1.0f);
        gamma.load(b.na.gamma, cols, t, 1.0f);
        if (SHIFT) beta.load(b.na.beta, cols, t, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VE;
            float o[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                o[e] = gamma.v[i][e] * S[0].v[i][e];
                if (SHIFT) o[e] += beta.v[i][e] * S[kSums - 1].v[i][e];
#pragma unroll
                for (int k = 0; k < kSums; ++k) A[WHOLE ? k : 0].v[i][e] += g.v[i][e] * S[k].v[i][e];
            }
            if (b.dgate && c < cols) store_vec<float, VE>(b.dgate + int64_t(group) * cols + c, o, cols - c);
        }
    }
    if constexpr (WHOLE) {
        if (b.part_a) leave(A, b.part_a + int64_t(blockIdx.x) * 2 * cols);
    }
    if (b.part_y) leave(Y, b.part_y + int64_t(blockIdx.x) * 2 * cols);
}

// The partial rows added up, 16 columns a workgroup, in an order that the sizes
// fix: workgroups of blockIdx.y = 0 those of the gates, of 1 those of N_y.  64
// groups of threads share a gate's runs where there are as many, elsewhere the
// gates.  (64 columns and 16 groups: 16 us at 4096 columns and 512 partial rows, and at
// 256 columns, which were four workgroups; so 8 and 5.)
constexpr uint32_t kAtOnce = 2;
constexpr int kSumCols = 16, kSumGroups = 64, kSumWaves = kSumCols * kSumGroups / 64;

struct Sums {
    const float *part_a, *part_y;
    const float *gate, *gamma_a, *beta_a;
    float *dgate, *dgamma_a, *dbeta_a, *dgamma_y, *dbeta_y;
    uint32_t groups, chunks, last, parts;  // last: runs of the last gate; parts: workgroups of the first pass
    int cols;
    bool whole, a, y, shift;  // part_a is of whole gates; asked for; the second sums are there
};

__global__ __launch_bounds__(kSumCols *kSumGroups) void residual_norm_sum_kernel(Sums s) {
    __shared__ float red[2][kSumWaves][kSumCols];
    const int lane = threadIdx.x & (kSumCols - 1), grp = threadIdx.x / kSumCols;
    const int64_t cols = s.cols, c = int64_t(blockIdx.x) * kSumCols + lane;
    const bool in = c < cols;
    // both sums of partial rows from, from + by .. of `count` from p on
    const auto run = [&](const float *p, uint32_t from, uint32_t count, uint32_t by, float (&v)[2])
        __attribute__((always_inline)) {
            v[0] = v[1] = 0.0f;
            if (!in) return;
#pragma unroll 8
            for (uint32_t k = from; k < count; k += by) {
                v[0] += p[int64_t(k) * 2 * cols + c];
                if (s.shift) v[1] += p[int64_t(k) * 2 * cols + cols + c];
            }
        };
    // v of all groups: a wavefront's four, then the wavefronts (every group gets it)
    const auto join = [&](float (&v)[2]) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int off = kSumCols; off < 64; off <<= 1) v[k] += __shfl_xor(v[k], off, 64);
        __syncthreads();
        if ((threadIdx.x & 63) < kSumCols) {
            red[0][threadIdx.x >> 6][lane] = v[0];
            red[1][threadIdx.x >> 6][lane] = v[1];
        }
        __syncthreads();
        v[0] = v[1] = 0.0f;
#pragma unroll
        for (int k = 0; k < kSumWaves; ++k) {
            v[0] += red[0][k][lane];
            v[1] += red[1][k][lane];
        }
    };
    float v[2];
    if (blockIdx.y == 1 ? !s.y : !s.a) return;
    if (blockIdx.y == 1 || s.whole) {
        run(blockIdx.y == 1 ? s.part_y : s.part_a, grp, s.parts, kSumGroups, v);
        join(v);
        float *to0 = blockIdx.y == 1 ? s.dgamma_y : s.dgamma_a, *to1 = blockIdx.y == 1 ? s.dbeta_y : s.dbeta_a;
        if (grp == 0 && in) {
            if (to0) to0[c] = v[0];
            if (to1) to1[c] = v[1];
        }
        return;
    }
    const float gamma = s.gamma_a && in ? s.gamma_a[c] : 1.0f, beta = s.beta_a && in ? s.beta_a[c] : 0.0f;
    float all[2] = {0.0f, 0.0f};
    const auto add = [&](uint32_t g, float gate, const float (&w)[2], bool write) __attribute__((always_inline)) {
        if (!in) return;
        if (s.dgate && write) s.dgate[int64_t(g) * cols + c] = gamma * w[0] + beta * w[1];
        all[0] += gate * w[0];
        all[1] += gate * w[1];
    };
    if (s.chunks >= uint32_t(kSumGroups)) {
        for (uint32_t g = 0; g < s.groups; ++g) {
            run(s.part_a + int64_t(g) * s.chunks * 2 * cols, grp, g + 1 < s.groups ? s.chunks : s.last, kSumGroups, v);
            const float gate = s.gate && in ? s.gate[int64_t(g) * cols + c] : 1.0f;
            join(v);
            add(g, gate, v, grp == 0);
        }
    } else {
        for (uint32_t g0 = grp; g0 < s.groups; g0 += kAtOnce * kSumGroups) {
            float w[kAtOnce][2], gate[kAtOnce];  // loads of several gates in flight
#pragma unroll
            for (uint32_t u = 0; u < kAtOnce; ++u) {
                const uint32_t g = min(g0 + u * kSumGroups, s.groups - 1);
                gate[u] = s.gate && in ? s.gate[int64_t(g) * cols + c] : 1.0f;
                run(s.part_a + int64_t(g) * s.chunks * 2 * cols, 0, g + 1 < s.groups ? s.chunks : s.last, 1, w[u]);
            }
#pragma unroll
            for (uint32_t u = 0; u < kAtOnce; ++u)
                if (g0 + u * kSumGroups < s.groups) add(g0 + u * kSumGroups, gate[u], w[u], true);
        }
        join(all);
    }
    if (grp == 0 && in) {
        if (s.dgamma_a) s.dgamma_a[c] = all[0];
        if (s.dbeta_a) s.dbeta_a[c] = all[1];
    }
}

// f(columns of a vector, threads per row, vectors per thread) for a row of cols columns: a part of a
// wavefront for short rows (32768 x 64 bfloat16 forward 9 us, in a wavefront a row 30;
// 25088 x 256 12 and 26), one while that takes few vectors a lane (no barrier), then the
// fewest wavefronts, of some numbers, that hold it in eight columns each, 16 wavefronts
// of sixteen columns above 8192 (4096 x 5120 bfloat16 in 640 threads a row 49 us forward
// and 57 backward, in 1024 59 and 74; 8192 x 2560 in 320 53 and 48, in 512 53 and 53).
// Backward, short rows of 16-bit types are held in four columns each, for eight and
// the vectors' sums are more than the registers of two workgroups on a compute unit
// (32768 x 64 12.7 against 19.5 us).
template <class T, bool BWD, class F>
void with_shape(int64_t cols, F &&f) {
    constexpr int VE = 16 / sizeof(T), kShort = BWD ? 4 : VE;
    constexpr bool kWide = VE == 8 && !BWD;
    const IntC<VE> ve;
    const IntC<kShort> few;
    const int64_t v = (cols + VE - 1) / VE, s = (cols + kShort - 1) / kShort;
    if (s <= 8) return f(few, IntC<8>{}, IntC<1>{});
    if (s <= 16) return f(few, IntC<16>{}, IntC<1>{});
    if (s <= 32) return f(few, IntC<32>{}, IntC<1>{});
    if (s <= 64) return f(few, IntC<64>{}, IntC<1>{});
    if (v <= 64) return f(ve, IntC<64>{}, IntC<1>{});
    if (v <= 128) return f(ve, IntC<kWide ? 128 : 64>{}, IntC<kWide ? 1 : 2>{});
    if constexpr (kWide) {
        if (v <= 192) return f(ve, IntC<192>{}, IntC<1>{});
    }
    if (v <= 256) return f(ve, IntC<256>{}, IntC<1>{});
    if constexpr (VE == 8) {
        if (v <= 320) return f(ve, IntC<320>{}, IntC<1>{});
        if (v <= 384) return f(ve, IntC<384>{}, IntC<1>{});
    }
    if (v <= 512) return f(ve, IntC<VE == 8 ? 512 : 256>{}, IntC<VE == 8 ? 1 : 2>{});
    if constexpr (VE == 8) {
        if (v <= 640) return f(ve, IntC<640>{}, IntC<1>{});
        if (v <= 768) return f(ve, IntC<768>{}, IntC<1>{});
    }
    if (v <= 1024) return f(ve, IntC<VE == 8 ? 1024 : 512>{}, IntC<VE == 8 ? 1 : 2>{});
    if (v <= 2048) return f(ve, IntC<1024>{}, IntC<2>{});
    if constexpr (VE == 4) f(ve, IntC<1024>{}, IntC<4>{});
}

// How the rows are cut for the backward pass: into as many runs as workgroups, by
// the rows that there are (a last gate of few rows counted as a whole one left every
// other workgroup without a run: 5000 x 2000 bfloat16, gates of 4000 rows, 37 us and 49;
// 8192 x 700 float32, gates of 8000, 43 and 66).
struct Runs {
    uint32_t groups, chunks, chunk_rows;
    uint32_t last;  // runs of the last gate, which may have fewer rows
    uint32_t units() const { return groups ? (groups - 1) * chunks + last : 0; }
    bool whole() const { return groups > uint32_t(kMaxGroups); }
};
Runs runs_of(int64_t rows, int64_t cols, int64_t gate_rows) {
    const int64_t groups = (rows + gate_rows - 1) / gate_rows, least = cols <= 1024 ? 8 : 4;
    const int64_t last_rows = rows - (groups - 1) * gate_rows;
    int64_t chunks = kMaxGroups * gate_rows / rows;
    if (chunks > (gate_rows + least - 1) / least) chunks = (gate_rows + least - 1) / least;
    for (;; --chunks) {
        if (chunks < 1) chunks = 1;
        const int64_t chunk_rows = (gate_rows + chunks - 1) / chunks, runs = (gate_rows + chunk_rows - 1) / chunk_rows;
        const Runs r{uint32_t(groups), uint32_t(runs), uint32_t(chunk_rows), uint32_t((last_rows + chunk_rows - 1) / chunk_rows)};
        if (chunks == 1 || r.units() <= uint32_t(kMaxGroups)) return r;
    }
}

bool sizes_ok(int64_t rows, int64_t cols) { return rows >= 0 && cols >= 0 && rows <= kMaxDim && cols <= kMaxCols; }

// Whether a tensor of `bytes` is another or lies apart from it.
bool same_or_apart(const void *a, const void *b, size_t bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return !a || !b || x == y || x + bytes <= y || y + bytes <= x;
}
bool apart(const void *a, const void *b, size_t bytes) { return !a || (a != b && same_or_apart(a, b, bytes)); }

bool kind_ok(int kind) { return kind == IONN_NORM_NONE || kind == IONN_NORM_LAYER || kind == IONN_NORM_RMS; }

}  // namespace
}  // namespace ionn

using namespace ionn;

extern "C" {

int ionn_residual_norm_fwd(const void *a, const void *x, int norm_a, const float *gamma_a, const float *beta_a,
                           const float *gate, int64_t gate_rows, double alpha, int norm_y, const float *gamma_y,
                           const float *beta_y, double eps, void *y, void *n, float *mean_a, float *rstd_a,
                           float *mean_y, float *rstd_y, int dtype, int64_t rows, int64_t cols, uint32_t *absmax_n,
                           void *stream) {
    clear_error();
    IONN_REQUIRE(dtype_ok(dtype), IONN_ERR_ARG, "ionn_residual_norm_fwd: dtype = %d", dtype);
    IONN_REQUIRE(kind_ok(norm_a) && kind_ok(norm_y), IONN_ERR_ARG, "ionn_residual_norm_fwd: norms %d and %d", norm_a,
                 norm_y);
    IONN_REQUIRE(sizes_ok(rows, cols), IONN_ERR_SHAPE, "ionn_residual_norm_fwd: rows = %lld, cols = %lld (at most %lld)",
                 (long long)rows, (long long)cols, (long long)kMaxCols);
    IONN_REQUIRE(eps >= 0.0 && eps <= 3.0e38 && alpha >= -3.0e38 && alpha <= 3.0e38, IONN_ERR_RANGE,
                 "ionn_residual_norm_fwd: eps = %g, alpha = %g", eps, alpha);
    IONN_REQUIRE(gate_rows >= 0 && gate_rows <= kMaxDim, IONN_ERR_RANGE, "ionn_residual_norm_fwd: gate_rows = %lld",
                 (long long)gate_rows);
    IONN_REQUIRE(norm_a != IONN_NORM_NONE || (!gamma_a && !beta_a && !mean_a && !rstd_a), IONN_ERR_ARG,
                 "ionn_residual_norm_fwd: parameters or statistics of no norm of a");
    IONN_REQUIRE(norm_y != IONN_NORM_NONE || (!n && !gamma_y && !beta_y && !mean_y && !rstd_y && !absmax_n), IONN_ERR_ARG,
                 "ionn_residual_norm_fwd: parameters or results of no norm of y");
    IONN_REQUIRE((norm_a == IONN_NORM_LAYER || (!beta_a && !mean_a)) && (norm_y == IONN_NORM_LAYER || (!beta_y && !mean_y)),
                 IONN_ERR_ARG, "ionn_residual_norm_fwd: only a layer norm has a mean and a beta");
    if (rows == 0 || cols == 0) return IONN_OK;
    IONN_REQUIRE(a || (norm_a == IONN_NORM_NONE && !gate), IONN_ERR_ARG,
                 "ionn_residual_norm_fwd: a norm or a gate of no block");
    IONN_REQUIRE(x && (y || n), IONN_ERR_ARG, "ionn_residual_norm_fwd: NULL tensor");
    IONN_REQUIRE(n || (!mean_y && !rstd_y && !absmax_n), IONN_ERR_ARG,
                 "ionn_residual_norm_fwd: results of a norm of y that is not asked for");
    const size_t es = dtype_size(dtype), bytes = size_t(rows) * cols * es;
    IONN_REQUIRE(aligned(a, es) && aligned(x, es) && aligned(y, es) && aligned(n, es) && aligned(gamma_a, 4) &&
                     aligned(beta_a, 4) && aligned(gate, 4) && aligned(gamma_y, 4) && aligned(beta_y, 4) &&
                     aligned(mean_a, 4) && aligned(rstd_a, 4) && aligned(mean_y, 4) && aligned(rstd_y, 4) &&
                     aligned(absmax_n, 4),
                 IONN_ERR_ALIGN, "ionn_residual_norm_fwd: tensors must be aligned to their element size");
    IONN_REQUIRE(apart(n, y, bytes) && same_or_apart(y, a, bytes) && same_or_apart(y, x, bytes) &&
                     same_or_apart(n, a, bytes) && same_or_apart(n, x, bytes),
                 IONN_ERR_ARG, "ionn_residual_norm_fwd: y and n may be a or x, but not overlap them or each other otherwise");
    const int64_t share = gate && gate_rows > 0 && gate_rows < rows ? gate_rows : rows;
    const Forward f{a, x, y, n, {norm_a, gamma_a, beta_a, mean_a, rstd_a}, {norm_y, gamma_y, beta_y, mean_y, rstd_y},
                    gate, rows, uint32_t(share), int(cols), float(alpha), float(eps), absmax_n, bytes >= kStreamBytes};
    with_dtype(dtype, [&](auto tag) {
        using T = decltype(tag);
        with_shape<T, false>(cols, [&](auto ve, auto tpr, auto nv) {
            constexpr int VE = decltype(ve)::value, TPR = decltype(tpr)::value, NV = decltype(nv)::value, kBlock = fwd_threads(TPR);
            // as many workgroups as are resident at once: rows are dealt out evenly
            int64_t blocks = (rows + kBlock / TPR - 1) / (kBlock / TPR);
            const int64_t most = int64_t(device_cus()) * (kBlock < 1024 ? 1024 / kBlock : 1);
            if (blocks > most) blocks = most;
            residual_norm_fwd_kernel<T, VE, TPR, NV><<<dim3(unsigned(blocks)), dim3(kBlock), 0, as_stream(stream)>>>(f);
        });
    });
    return check_launch("ionn_residual_norm_fwd");
}

size_t ionn_residual_norm_bwd_workspace_bytes(int64_t rows, int64_t cols, int64_t gate_rows) {
    if (!sizes_ok(rows, cols) || gate_rows < 0 || gate_rows > kMaxDim || rows == 0 || cols == 0) return 0;
    const int64_t share = gate_rows > 0 && gate_rows < rows ? gate_rows : rows;
    size_t most = 0;
    for (int64_t s : {share, rows}) {  // (without a gate gate_rows does not count)
        const Runs r = runs_of(rows, cols, s);
        const size_t n = r.whole() ? uint32_t(kMaxGroups) : r.units();
        most = n > most ? n : most;
    }
    return (most + kMaxGroups) * 2 * size_t(cols) * sizeof(float);
}

int ionn_residual_norm_bwd(const void *dy, const void *dn, const void *a, const void *y, int norm_a,
                           const float *gamma_a, const float *beta_a, const float *gate, int64_t gate_rows, double alpha,
                           int norm_y, const float *gamma_y, const float *mean_a, const float *rstd_a,
                           const float *mean_y, const float *rstd_y, void *da, void *dx, float *dgamma_a, float *dbeta_a,
                           float *dgate, float *dgamma_y, float *dbeta_y, int dtype, int64_t rows, int64_t cols,
                           void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    IONN_REQUIRE(dtype_ok(dtype), IONN_ERR_ARG, "ionn_residual_norm_bwd: dtype = %d", dtype);
    IONN_REQUIRE(kind_ok(norm_a) && kind_ok(norm_y), IONN_ERR_ARG, "ionn_residual_norm_bwd: norms %d and %d", norm_a,
                 norm_y);
    IONN_REQUIRE(sizes_ok(rows, cols), IONN_ERR_SHAPE, "ionn_residual_norm_bwd: rows = %lld, cols = %lld (at most %lld)",
                 (long long)rows, (long long)cols, (long long)kMaxCols);
    IONN_REQUIRE(alpha >= -3.0e38 && alpha <= 3.0e38, IONN_ERR_RANGE, "ionn_residual_norm_bwd: alpha = %g", alpha);
    IONN_REQUIRE(gate_rows >= 0 && gate_rows <= kMaxDim, IONN_ERR_RANGE, "ionn_residual_norm_bwd: gate_rows = %lld",
                 (long long)gate_rows);
    const bool sums_a = dgamma_a || dbeta_a || dgate, sums_y = dgamma_y || dbeta_y;
    IONN_REQUIRE(norm_a != IONN_NORM_NONE || (!gamma_a && !beta_a && !mean_a && !rstd_a && !dgamma_a && !dbeta_a),
                 IONN_ERR_ARG, "ionn_residual_norm_bwd: parameters or gradients of no norm of a");
    IONN_REQUIRE(norm_y != IONN_NORM_NONE || (!dn && !gamma_y && !mean_y && !rstd_y && !sums_y), IONN_ERR_ARG,
                 "ionn_residual_norm_bwd: parameters or gradients of no norm of y");
    IONN_REQUIRE((norm_a == IONN_NORM_LAYER || (!beta_a && !mean_a && !dbeta_a)) &&
                     (norm_y == IONN_NORM_LAYER || (!mean_y && !dbeta_y)),
                 IONN_ERR_ARG, "ionn_residual_norm_bwd: only a layer norm has a mean and a beta");
    IONN_REQUIRE(gate || !dgate, IONN_ERR_ARG, "ionn_residual_norm_bwd: dgate of no gate");
    if (cols == 0) return IONN_OK;
    const bool some = rows > 0;
    IONN_REQUIRE(!some || ((dy || dn) && (da || dx || sums_a || sums_y)), IONN_ERR_ARG,
                 "ionn_residual_norm_bwd: no error, or nothing to compute");
    IONN_REQUIRE(!some || norm_y == IONN_NORM_NONE ||
                     (dn && y && rstd_y && (mean_y || norm_y == IONN_NORM_RMS)),
                 IONN_ERR_ARG, "ionn_residual_norm_bwd: the norm of y needs dn, y and its statistics");
    IONN_REQUIRE(!some || (a ? norm_a == IONN_NORM_NONE || (rstd_a && (mean_a || norm_a == IONN_NORM_RMS))
                             : !da && !sums_a && !gate && norm_a == IONN_NORM_NONE),
                 IONN_ERR_ARG, "ionn_residual_norm_bwd: a's gradients need a and its statistics");
    const size_t es = dtype_size(dtype), bytes = size_t(rows) * cols * es;
    IONN_REQUIRE(aligned(dy, es) && aligned(dn, es) && aligned(a, es) && aligned(y, es) && aligned(da, es) &&
                     aligned(dx, es) && aligned(gamma_a, 4) && aligned(beta_a, 4) && aligned(gate, 4) &&
                     aligned(gamma_y, 4) && aligned(mean_a, 4) && aligned(rstd_a, 4) && aligned(mean_y, 4) &&
                     aligned(rstd_y, 4) && aligned(dgamma_a, 4) && aligned(dbeta_a, 4) && aligned(dgate, 4) &&
                     aligned(dgamma_y, 4) && aligned(dbeta_y, 4),
                 IONN_ERR_ALIGN, "ionn_residual_norm_bwd: tensors must be aligned to their element size");
    IONN_REQUIRE(!some || apart(da, dx, bytes), IONN_ERR_ARG, "ionn_residual_norm_bwd: da and dx overlap");
    for (const void *in : {dy, dn, a, y})
        IONN_REQUIRE(!some || (same_or_apart(da, in, bytes) && same_or_apart(dx, in, bytes)), IONN_ERR_ARG,
                     "ionn_residual_norm_bwd: da and dx may be an input, but not overlap one in part");
    const int64_t share = gate && gate_rows > 0 && gate_rows < rows ? gate_rows : rows;
    const size_t need = ionn_residual_norm_bwd_workspace_bytes(rows, cols, gate_rows);
    IONN_REQUIRE(!(sums_a || sums_y) || need == 0 || (workspace && aligned(workspace, 16) && workspace_bytes >= need),
                 IONN_ERR_WORKSPACE, "ionn_residual_norm_bwd: needs a 16-byte aligned workspace of %zu bytes", need);
    hipStream_t st = as_stream(stream);
    if (!some) {  // (no rows: one gate of all of them)
        for (float *v : {dgamma_a, dbeta_a, dgate, dgamma_y, dbeta_y}) zero_bytes(v, cols * 4, st);
        return check_launch("ionn_residual_norm_bwd");
    }
    const Runs runs = runs_of(rows, cols, share);
    int64_t blocks = 0;
    float *part_a = sums_a ? static_cast<float *>(workspace) : nullptr;
    float *part_y = nullptr;
    if (sums_y)
        part_y = static_cast<float *>(workspace) + size_t(runs.whole() ? uint32_t(kMaxGroups) : runs.units()) * 2 * cols;
    const Backward b{dy, dn, a, y, da, dx,
                     {norm_a, gamma_a, beta_a, const_cast<float *>(mean_a), const_cast<float *>(rstd_a)},
                     {norm_y, gamma_y, nullptr, const_cast<float *>(mean_y), const_cast<float *>(rstd_y)},
                     gate, rows, uint32_t(share), runs.chunks, runs.chunk_rows, runs.units(), int(cols), float(alpha),
                     part_a, part_y, dgate, bytes >= kStreamBytes};
    with_dtype(dtype, [&](auto tag) {
        using T = decltype(tag);
        with_shape<T, true>(cols, [&](auto ve, auto tpr, auto nv) {
            constexpr int VE = decltype(ve)::value, TPR = decltype(tpr)::value, NV = decltype(nv)::value, kBlock = bwd_threads(TPR);
            const int64_t each = runs.whole() ? kBlock / TPR : 1;
            blocks = (runs.units() + each - 1) / each;
            if (blocks > kMaxGroups) blocks = kMaxGroups;
            const dim3 grid{unsigned(blocks)}, block{unsigned(kBlock)};
            const auto launch = [&](auto whole, auto shift) {
                residual_norm_bwd_kernel<T, VE, TPR, NV, decltype(whole)::value, decltype(shift)::value>
                    <<<grid, block, 0, st>>>(b);
            };
            const bool shift = norm_a == IONN_NORM_LAYER || norm_y == IONN_NORM_LAYER;
            if (runs.whole()) shift ? launch(IntC<1>{}, IntC<1>{}) : launch(IntC<1>{}, IntC<0>{});
            else shift ? launch(IntC<0>{}, IntC<1>{}) : launch(IntC<0>{}, IntC<0>{});
        });
    });
    if (int rc = check_launch("ionn_residual_norm_bwd")) return rc;
    if (sums_a || sums_y) {
        const Sums s{part_a, part_y, gate, gamma_a, beta_a, dgate, dgamma_a, dbeta_a, dgamma_y, dbeta_y,
                     runs.groups, runs.chunks, runs.last, uint32_t(blocks), int(cols), runs.whole(), sums_a, sums_y,
                     norm_a == IONN_NORM_LAYER || norm_y == IONN_NORM_LAYER};
        residual_norm_sum_kernel<<<dim3(unsigned((cols + kSumCols - 1) / kSumCols), 2), dim3(kSumCols * kSumGroups), 0, st>>>(s);
        return check_launch("ionn_residual_norm_bwd");
    }
    return IONN_OK;
}

}  // extern "C"
