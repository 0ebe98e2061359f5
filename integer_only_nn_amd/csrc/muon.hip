// The Muon step: momentum, the update orthogonalised by Newton-Schulz products,
// and the weights, in place.
//
//   M = mu M + g,  u = g + mu M (nesterov) or M,  X = u / (|u| + eps)
//   k times:  A = X X^T,  X = a X + (b A + c A A) X
//   P = P (1 - lr wd) - lr scale X
//
// The products are the work: k (3 m^2 n + m^3) operations for the m x n matrix
// laid with its shorter side first (a tall one is transposed), A and A A being
// symmetric.  They run on the float16 matrix cores with every operand as a pair of
// float16 terms (muon_tile.h): 22 bits, for P and M are float32, and one term
// alone would leave X off by 1.5e-3 of its size, one of bfloat16 by 1.2e-2
// (where a few directions dominate, ten times as much).  Scaled by 2^12, which
// keeps the terms of entries down to 2^-26 of a singular value's size out of
// float16's subnormal range and the largest (|b| + |c| of B) a factor of 5 below
// its largest value.
//
// A product leaves its sums in pieces, and the pass after it adds them, applies
// the polynomial and writes pairs: for a symmetric matrix both of its halves from
// the lower tiles, for X both X and X^T, so that each operand is K-major, and at
// the end P.  Matrices of a batch share every launch.
#include "muon_tile.h"

#include <cmath>

namespace ionn {
namespace {

using muon::v16f;
using muon::v4f;
using muon::Work;

constexpr int kTable = 8;  // matrices of a launch
constexpr int kThreads = 256;
constexpr int kSumBlocks = 256;  // workgroups of a matrix that take |u|
constexpr float kScale = 4096.0f;
constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr int64_t kMaxElements = int64_t(1) << 28;  // of the padded matrix: its pairs stay below 2^30 bytes

struct Mat {
    float *P, *M;
    const void *G;
    int8_t *X, *XT, *A, *B;  // pairs: [mp][np], [np][mp], [mp][mp], [mp][mp]
    double *sums;            // [blocks]
    float *part;
    int64_t count;
    int m, n, mp, np;
    int cols;   // of P: n, or m where the matrix is tall
    int tall;
    int blocks;  // partial sums of |u|^2
    float scale;
};

enum Product { XX = 0, AA = 1, BX = 2 };

struct Table {
    Mat mat[kTable];
    int first[kTable + 1];  // of a launch's workgroups or wavefronts
    int L;
};

struct Hyper {
    float mu, eps;
    double lr, wd;
    int nesterov;
    const float *lr_dev, *grad_scale;
    uint32_t *absmax;
};

__device__ __forceinline__ int find(const Table &t, int id) {
    int l = 0;
    while (l + 1 < t.L && id >= t.first[l + 1]) ++l;
    return l;
}

__device__ __forceinline__ float update_of(float m, float g, const Hyper &h) { return h.nesterov ? fmaf(h.mu, m, g) : m; }

// M = mu M + g, and each workgroup's sum of u^2 (in float64: float32 squares leave
// their range at 1e19 and 1e-23).
template <class T>
__global__ __launch_bounds__(kThreads) void momentum_kernel(Table t, Hyper h) {
    __shared__ double red[kThreads / 64];
    const int l = find(t, int(blockIdx.x)), b = int(blockIdx.x) - t.first[l];
    const Mat &a = t.mat[l];
    const T *G = static_cast<const T *>(a.G);
    const float gs = h.grad_scale ? *h.grad_scale : 1.0f;
    double s = 0.0;
    for (int64_t i = (int64_t(b) * kThreads + threadIdx.x) * 4; i < a.count; i += int64_t(a.blocks) * kThreads * 4) {
        const int valid = int(a.count - i < 4 ? a.count - i : 4);
        const auto g = load_raw<T, 4>(G + i, valid);
        const auto m = load_raw<float, 4>(a.M + i, valid);
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = float(g[e]) * gs;
            o[e] = fmaf(h.mu, m[e], x);
            const double u = e < valid ? double(update_of(o[e], x, h)) : 0.0;
            s += u * u;
        }
        store_vec<float, 4>(a.M + i, o, valid);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) a.sums[b] = (red[0] + red[1]) + (red[2] + red[3]);
}

// ---- blocks of 32 x 32 ---------------------------------------------------------
// A lane holds row lane % 32, columns 8 q + 4 (lane / 32) .. + 3 in v[4 q ..], as
// the matrix instructions leave them.

typedef _Float16 v4h __attribute__((ext_vector_type(4)));

// Where a lane's values of block (r0, c0) lie in a matrix of pairs with rows of K.
__device__ __forceinline__ _Float16 *pair_at(int8_t *base, int K, int r0, int c0, int lane) {
    return reinterpret_cast<_Float16 *>(base) + int64_t(r0 + (lane & 31)) * 2 * K + 2 * c0 + 4 * (lane >> 5);
}

__device__ __forceinline__ void store_pairs(int8_t *base, int K, int r0, int c0, int lane, const float (&v)[16]) {
    _Float16 *p = pair_at(base, K, r0, c0, lane);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v4h hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = _Float16(v[4 * q + e]);
            lo[e] = _Float16(v[4 * q + e] - float(hi[e]));
        }
        *reinterpret_cast<v4h *>(p + 8 * q) = hi;
        *reinterpret_cast<v4h *>(p + 8 * q + 32) = lo;
    }
}

__device__ __forceinline__ void load_pairs(int8_t *base, int K, int r0, int c0, int lane, float (&v)[16]) {
    const _Float16 *p = pair_at(base, K, r0, c0, lane);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const v4h hi = *reinterpret_cast<const v4h *>(p + 8 * q), lo = *reinterpret_cast<const v4h *>(p + 8 * q + 32);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * q + e] = float(hi[e]) + float(lo[e]);
    }
}

// The block's transpose, through a wavefront's own LDS.
__device__ __forceinline__ void transpose(float (&v)[16], float (*buf)[33], int lane) {
    const int r = lane & 31, c = 4 * (lane >> 5);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) buf[r][8 * q + c + e] = v[4 * q + e];
    dfp8::in_order();
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * q + e] = buf[8 * q + c + e][r];
    dfp8::in_order();
}

// X = u / (|u| + eps) and X^T as pairs, zeros in the padding: a wavefront a block
// of u (of P's layout).
template <class T>
__global__ __launch_bounds__(kThreads) void scale_kernel(Table t, Hyper h) {
    __shared__ float buf[kThreads / 64][32][33];
    __shared__ double red[kThreads / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l = find(t, int(blockIdx.x));
    const Mat &a = t.mat[l];
    double s = 0.0;
    for (int i = threadIdx.x; i < a.blocks; i += kThreads) s += a.sums[i];
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
    if (lane == 0) red[wave] = s;
    __syncthreads();
    s = (red[0] + red[1]) + (red[2] + red[3]);
    const double norm = sqrt(s) + double(h.eps);
    const double factor = norm > 0.0 ? double(kScale) / norm : (norm == 0.0 ? 0.0 : norm);  // (NaN stays one)
    // rows and columns of P, and of its padded form
    const int rows = a.tall ? a.n : a.m, cols = a.cols, rp = a.tall ? a.np : a.mp, cp = a.tall ? a.mp : a.np;
    const int across = cp / 32, b = (int(blockIdx.x) - t.first[l]) * (kThreads / 64) + wave;
    const int r0 = 32 * (b / across), c0 = 32 * (b % across);
    if (r0 >= rp) return;
    const int r = r0 + (lane & 31);
    const T *G = static_cast<const T *>(a.G);
    const float gs = h.grad_scale ? *h.grad_scale : 1.0f;
    float v[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int c = c0 + 8 * q + 4 * (lane >> 5), valid = r < rows ? cols - c : 0;
        const int64_t at = int64_t(r) * cols + c;
        const auto m = load_raw<float, 4>(a.M + at, valid);
        typename Vec<T, 4>::type g = load_raw<T, 4>(G + at, h.nesterov ? valid : 0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[4 * q + e] = e < valid ? float(double(update_of(m[e], float(g[e]) * gs, h)) * factor) : 0.0f;
    }
    store_pairs(a.tall ? a.XT : a.X, cp, r0, c0, lane, v);
    transpose(v, buf[wave], lane);
    store_pairs(a.tall ? a.X : a.XT, rp, c0, r0, lane, v);
}

// ---- products ------------------------------------------------------------------

// chunk: of all products of a launch.
template <int SIDE>
__host__ __device__ __forceinline__ Work work_of(const Mat &a, int product, int chunk) {
    Work w;
    w.A = product == XX ? a.X : product == AA ? a.A : a.B;
    w.B = product == XX ? a.X : product == AA ? a.A : a.XT;
    w.part = a.part;
    w.rows = a.mp;
    w.cols = product == BX ? a.np : a.mp;
    w.K = product == XX ? a.np : a.mp;
    w.tri = product != BX;
    const int tm = w.rows / SIDE, tn = w.cols / SIDE;
    w.tiles = w.tri ? tm * (tm + 1) / 2 : tm * tn;
    w.S = w.K / 64;
    w.chunk = chunk;
    w.slots = (chunk + w.S - 1) / w.S + 1;
    w.groups = int((int64_t(w.tiles) * w.S + chunk - 1) / chunk);
    return w;
}

__global__ __launch_bounds__(kThreads) void product128_kernel(Table t, int product, int chunk) {
    __shared__ __attribute__((aligned(1024))) int8_t lds[dfp8::kStages * dfp8::kStage128];
    const int l = find(t, int(blockIdx.x));
    const Work w = work_of<128>(t.mat[l], product, chunk);
    muon::pieces<128>(w, int(blockIdx.x) - t.first[l], [&](int ti, int tj, int k0, int k1, float *to) {
        muon::piece128(w, ti, tj, k0, k1, to, lds);
    });
}

__global__ __launch_bounds__(g256::NT, 1) void product256_kernel(Mat a, int product, int chunk) {
    __shared__ __attribute__((aligned(1024))) int8_t sA0[g256::TILE_BYTES];
    __shared__ __attribute__((aligned(1024))) int8_t sB0[g256::TILE_BYTES];
    __shared__ __attribute__((aligned(1024))) int8_t sA1[g256::TILE_BYTES];
    __shared__ __attribute__((aligned(1024))) int8_t sB1[g256::TILE_BYTES];
    const Work w = work_of<256>(a, product, chunk);
    // neighbouring runs on one XCD
    int g = int(blockIdx.x);
    if (w.groups % 8 == 0) g = (g % 8) * (w.groups / 8) + g / 8;
    muon::pieces<256>(w, g, [&](int ti, int tj, int k0, int k1, float *to) {
        muon::piece256(w, ti, tj, k0, k1, to, sA0, sB0, sA1, sB1);
    });
}

// What follows a product: a wavefront a block of 32 x 32.
template <int SIDE>
__global__ __launch_bounds__(kThreads) void finish_kernel(Table t, Hyper h, int product, int chunk, int last) {
    constexpr int F = SIDE / 64, kBlocks = (SIDE / 32) * (SIDE / 32);  // of a wavefront's side; of a tile
    __shared__ float buf[kThreads / 64][32][33];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l = find(t, int(blockIdx.x));
    const Mat &a = t.mat[l];
    const Work w = work_of<SIDE>(a, product, chunk);
    const int id = (int(blockIdx.x) - t.first[l]) * (kThreads / 64) + wave;
    const int tile = id / kBlocks, k = id % kBlocks;  // k: [wavefront][i][j] of the slot
    uint32_t top = 0;
    if (tile < w.tiles) {
        int ti, tj;
        muon::tile_at(w, SIDE, tile, ti, tj);
        const int part = k / (F * F), i = k % (F * F) / F, j = k % F;
        const int r0 = SIDE * ti + (SIDE / 2) * (part >> 1) + 32 * i, c0 = SIDE * tj + (SIDE / 2) * (part & 1) + 32 * j;
        float v[16] = {};
        const int first = tile * w.S / chunk, end = ((tile + 1) * w.S - 1) / chunk;
        for (int g = first; g <= end; ++g) {
            const int slot = tile - g * chunk / w.S;
            const v4f *p = reinterpret_cast<const v4f *>(w.part + (int64_t(g) * w.slots + slot) * (SIDE * SIDE)) +
                           (k * 4) * 64 + lane;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const v4f s = p[64 * q];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * q + e] += s[e];
            }
        }
        float x[16];
        if (product == AA) load_pairs(a.A, a.mp, r0, c0, lane, x);
        if (product == BX) load_pairs(a.X, a.np, r0, c0, lane, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            v[e] *= 1.0f / kScale;
            if (product == AA) v[e] = fmaf(kC, v[e], kB * x[e]);
            if (product == BX) v[e] = fmaf(kA, x[e], v[e]);
        }
        if (product != BX) {
            int8_t *to = product == XX ? a.A : a.B;
            store_pairs(to, a.mp, r0, c0, lane, v);
            if (ti != tj) {
                transpose(v, buf[wave], lane);
                store_pairs(to, a.mp, c0, r0, lane, v);
            }
        } else if (!last) {
            store_pairs(a.X, a.np, r0, c0, lane, v);
            transpose(v, buf[wave], lane);
            store_pairs(a.XT, a.mp, c0, r0, lane, v);
        } else {
            if (a.tall) transpose(v, buf[wave], lane);
            const int pr = (a.tall ? c0 : r0) + (lane & 31), pc = (a.tall ? r0 : c0) + 4 * (lane >> 5);
            const int rows = a.tall ? a.n : a.m, cols = a.cols;
            const double lr = h.lr_dev ? double(*h.lr_dev) : h.lr;
            const float keep = float(1.0 - lr * h.wd), rate = float(lr * double(a.scale) / double(kScale));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = pc + 8 * q, valid = pr < rows ? cols - c : 0;
                if (valid <= 0) continue;
                float *p = a.P + int64_t(pr) * cols + c;
                const auto old = load_raw<float, 4>(p, valid);
                float o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    o[e] = old[e] * keep - v[4 * q + e] * rate;
                    if (e < valid) top = max(top, mag_bits(o[e]));
                }
                store_vec<float, 4>(p, o, valid);
            }
        }
    }
    if (last && h.absmax) {
        top = wave_max_u32(top);
        if (lane == 0) publish_max_u32(h.absmax + l, top);
    }
}

// ---- host ------------------------------------------------------------------------

int64_t up(int64_t a, int64_t to) { return (a + to - 1) / to * to; }

// Whether a matrix is worked in tiles of 256, by itself, rather than in tiles of
// 128 with others.
bool large(int64_t m, int64_t n) { return up(m, 256) * up(n, 256) >= int64_t(64) * 256 * 256; }

// The run of double steps that each workgroup takes of a product, over all
// matrices of a launch: one workgroup per compute unit and 256 x 256 tile, two and
// 128 x 128, but none of fewer than four double steps.
int chunk_of(int64_t total, int groups) {
    const int64_t c = (total + groups - 1) / groups;
    return int(c < 4 ? 4 : c);
}

struct Layout {
    int side;
    int chunk[3];
    size_t bytes;
};

// Lays the matrices of a batch out in one workspace (base may be NULL for the bytes alone).
Layout lay_out(Mat *mats, int L, char *base) {
    Layout y{large(mats[0].m, mats[0].n) ? 256 : 128, {}, 0};
    const auto take = [&](size_t bytes) {
        char *p = base ? base + y.bytes : nullptr;
        y.bytes += size_t(up(int64_t(bytes), 1024));
        return p;
    };
    for (int l = 0; l < L; ++l) {
        Mat &a = mats[l];
        a.mp = int(up(a.m, y.side));
        a.np = int(up(a.n, y.side));
        const size_t x = size_t(a.mp) * a.np * 4, s = size_t(a.mp) * a.mp * 4;
        a.X = reinterpret_cast<int8_t *>(take(x));
        a.XT = reinterpret_cast<int8_t *>(take(x));
        a.A = reinterpret_cast<int8_t *>(take(s));
        a.B = reinterpret_cast<int8_t *>(take(s));
        a.sums = reinterpret_cast<double *>(take(kSumBlocks * sizeof(double)));
    }
    size_t most[kTable] = {};
    for (int p = 0; p < 3; ++p) {
        int64_t total = 0;
        const auto work = [&](int l, int chunk) {
            return y.side == 256 ? work_of<256>(mats[l], p, chunk) : work_of<128>(mats[l], p, chunk);
        };
        for (int l = 0; l < L; ++l) {
            const Work w = work(l, 1);
            total += int64_t(w.tiles) * w.S;
        }
        y.chunk[p] = chunk_of(total, y.side == 256 ? 256 : 512);
        for (int l = 0; l < L; ++l) {
            const Work w = work(l, y.chunk[p]);
            const size_t b = size_t(w.groups) * w.slots * y.side * y.side * sizeof(float);
            most[l] = b > most[l] ? b : most[l];
        }
    }
    for (int l = 0; l < L; ++l) mats[l].part = reinterpret_cast<float *>(take(most[l]));
    return y;
}

Mat mat_of(int64_t rows, int64_t cols) {
    Mat a{};
    a.tall = rows > cols;
    a.m = int(a.tall ? cols : rows);
    a.n = int(a.tall ? rows : cols);
    a.cols = int(cols);
    a.count = rows * cols;
    const int64_t b = (a.count + kThreads * 16 - 1) / (kThreads * 16);
    a.blocks = int(b < kSumBlocks ? b : kSumBlocks);
    return a;
}

bool size_ok(int64_t rows, int64_t cols) {
    return rows >= 1 && cols >= 1 && rows <= kMaxElements && cols <= kMaxElements &&
           up(rows, 256) * up(cols, 256) <= kMaxElements;
}

// Matrices from l on that share their launches.
int batch_of(int L, const int64_t *rows, const int64_t *cols, int l) {
    const auto m = [&](int i) { return rows[i] < cols[i] ? rows[i] : cols[i]; };
    const auto n = [&](int i) { return rows[i] < cols[i] ? cols[i] : rows[i]; };
    if (large(m(l), n(l))) return 1;
    int k = 1;
    while (k < kTable && l + k < L && !large(m(l + k), n(l + k))) ++k;
    return k;
}

template <int SIDE>
void launch_product(Table &t, const Hyper &h, const Layout &y, int p, bool last, hipStream_t st) {
    int groups = 0;
    for (int l = 0; l < t.L; ++l) {
        t.first[l] = groups;
        groups += work_of<SIDE>(t.mat[l], p, y.chunk[p]).groups;
    }
    t.first[t.L] = groups;
    if (SIDE == 256) product256_kernel<<<dim3(unsigned(groups)), dim3(g256::NT), 0, st>>>(t.mat[0], p, y.chunk[p]);
    else product128_kernel<<<dim3(unsigned(groups)), dim3(kThreads), 0, st>>>(t, p, y.chunk[p]);
    constexpr int kBlocks = (SIDE / 32) * (SIDE / 32) / (kThreads / 64);  // workgroups of a tile
    groups = 0;
    for (int l = 0; l < t.L; ++l) {
        t.first[l] = groups;
        groups += work_of<SIDE>(t.mat[l], p, y.chunk[p]).tiles * kBlocks;
    }
    t.first[t.L] = groups;
    finish_kernel<SIDE><<<dim3(unsigned(groups)), dim3(kThreads), 0, st>>>(t, h, p, y.chunk[p], last);
}

}  // namespace
}  // namespace ionn

using namespace ionn;

extern "C" {

size_t ionn_muon_workspace_bytes(int L, const int64_t *rows, const int64_t *cols) {
    if (L < 1 || !rows || !cols) return 0;
    for (int l = 0; l < L; ++l)
        if (!size_ok(rows[l], cols[l])) return 0;
    size_t most = 0;
    for (int l = 0; l < L;) {
        const int k = batch_of(L, rows, cols, l);
        Mat mats[kTable];
        for (int i = 0; i < k; ++i) mats[i] = mat_of(rows[l + i], cols[l + i]);
        const Layout y = lay_out(mats, k, nullptr);
        most = y.bytes > most ? y.bytes : most;
        l += k;
    }
    return most;
}

int ionn_muon_step(int L, float *const *P, const void *const *G, int g_dtype, float *const *M, const int64_t *rows,
                   const int64_t *cols, double lr, double momentum, int nesterov, double eps, double weight_decay,
                   int ns_steps, const double *scale, const float *lr_dev, const float *grad_scale, uint32_t *absmax_P,
                   void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    IONN_REQUIRE(L >= 1, IONN_ERR_SHAPE, "ionn_muon_step: L = %d < 1", L);
    IONN_REQUIRE(dtype_ok(g_dtype), IONN_ERR_ARG, "ionn_muon_step: g_dtype = %d", g_dtype);
    IONN_REQUIRE(P && G && M && rows && cols, IONN_ERR_ARG, "ionn_muon_step: NULL array");
    IONN_REQUIRE(momentum >= 0.0 && momentum < 1.0, IONN_ERR_RANGE, "ionn_muon_step: momentum = %g outside [0, 1)", momentum);
    IONN_REQUIRE(eps >= 0.0 && eps <= 3.0e38 && lr >= -3.0e38 && lr <= 3.0e38 && weight_decay >= -3.0e38 &&
                     weight_decay <= 3.0e38,
                 IONN_ERR_RANGE, "ionn_muon_step: eps = %g, lr = %g, weight_decay = %g", eps, lr, weight_decay);
    IONN_REQUIRE(ns_steps >= 1 && ns_steps <= 32, IONN_ERR_RANGE, "ionn_muon_step: ns_steps = %d outside [1, 32]", ns_steps);
    IONN_REQUIRE(aligned(lr_dev, 4) && aligned(grad_scale, 4) && aligned(absmax_P, 4), IONN_ERR_ALIGN,
                 "ionn_muon_step: device scalars must be 4-byte aligned");
    for (int l = 0; l < L; ++l) {
        IONN_REQUIRE(size_ok(rows[l], cols[l]), IONN_ERR_SHAPE, "ionn_muon_step: matrix %d is %lld x %lld", l,
                     (long long)rows[l], (long long)cols[l]);
        IONN_REQUIRE(P[l] && G[l] && M[l], IONN_ERR_ARG, "ionn_muon_step: matrix %d has a NULL pointer", l);
        IONN_REQUIRE(aligned(P[l], 4) && aligned(M[l], 4) && aligned(G[l], dtype_size(g_dtype)), IONN_ERR_ALIGN,
                     "ionn_muon_step: matrix %d must be aligned to its element size", l);
        IONN_REQUIRE(!scale || (scale[l] >= -3.0e38 && scale[l] <= 3.0e38), IONN_ERR_RANGE,
                     "ionn_muon_step: scale %d is %g", l, scale ? scale[l] : 0.0);
    }
    const size_t need = ionn_muon_workspace_bytes(L, rows, cols);
    IONN_REQUIRE(workspace && aligned(workspace, 256) && workspace_bytes >= need, IONN_ERR_WORKSPACE,
                 "ionn_muon_step: needs a 256-byte aligned workspace of %zu bytes", need);
    hipStream_t st = as_stream(stream);
    for (int l = 0; l < L;) {
        Table t{};
        t.L = batch_of(L, rows, cols, l);
        for (int i = 0; i < t.L; ++i) {
            Mat &a = t.mat[i];
            a = mat_of(rows[l + i], cols[l + i]);
            a.P = P[l + i];
            a.M = M[l + i];
            a.G = G[l + i];
            const double tall = double(rows[l + i]) / double(cols[l + i]);
            a.scale = float(scale ? scale[l + i] : (tall > 1.0 ? std::sqrt(tall) : 1.0));
        }
        const Layout y = lay_out(t.mat, t.L, static_cast<char *>(workspace));
        const Hyper h{float(momentum), float(eps), lr, weight_decay, nesterov, lr_dev, grad_scale,
                      absmax_P ? absmax_P + l : nullptr};
        int blocks = 0;
        for (int i = 0; i < t.L; ++i) {
            t.first[i] = blocks;
            blocks += t.mat[i].blocks;
        }
        t.first[t.L] = blocks;
        with_dtype(g_dtype, [&](auto tag) {
            momentum_kernel<decltype(tag)><<<dim3(unsigned(blocks)), dim3(kThreads), 0, st>>>(t, h);
        });
        blocks = 0;
        for (int i = 0; i < t.L; ++i) {
            t.first[i] = blocks;
            blocks += (t.mat[i].mp / 32) * (t.mat[i].np / 32) / (kThreads / 64);
        }
        t.first[t.L] = blocks;
        with_dtype(g_dtype, [&](auto tag) {
            scale_kernel<decltype(tag)><<<dim3(unsigned(blocks)), dim3(kThreads), 0, st>>>(t, h);
        });
        for (int k = 0; k < ns_steps; ++k)
            for (int p = 0; p < 3; ++p) {
                const bool last = p == BX && k + 1 == ns_steps;
                if (y.side == 256) launch_product<256>(t, h, y, p, last, st);
                else launch_product<128>(t, h, y, p, last, st);
            }
        if (int rc = check_launch("ionn_muon_step")) return rc;
        l += t.L;
    }
    return IONN_OK;
}

}  // extern "C"
