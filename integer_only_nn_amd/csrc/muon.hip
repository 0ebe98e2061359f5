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
// keeps the high terms of entries down to 2^-26 of a singular value's size out of
// float16's subnormal range and the largest entries, 2.8 of b A + c A A, a factor of
// 5 below its largest value.
// Steps are 2^-36 at least all the same: an X of 1e-3 (|u| a thousandth of eps), 2048 x
// 2048, is off by 9e-6 of itself, one of 1e-6 by 9e-3.
//
// A product leaves its sums in pieces, and the pass after it adds them, applies
// the polynomial and writes pairs: for a symmetric matrix both of its halves from
// the lower tiles, for X both X and X^T, so that each operand is K-major, and at
// the end P.  Small tiles do both in one launch.  Matrices of a batch share every
// launch.
//
// Measured: 4096 x 4096, bfloat16 gradients, 3.84 ms a step (3.77 to 4.28 by the card's
// clocks): of each of the five rounds 171 us for each symmetric product and 307 for
// X's (1280 and 1340 TFLOP/s of float16; the library's float16 product reaches
// 1373), 31 and 49 us for what follows them (168 to 268 MB, at the rate of a copy),
// and 29 and 49 us for the momentum and the first X.  1024 x 4096 470 us, 512 x 512
// 92, 64 x 64 56: 17 launches of 3.3 us, of which an empty one takes 2.1.
#include "muon_tile.h"

#include <climits>
#include <cmath>

namespace ionn {
namespace {

using muon::v16f;
using muon::v4f;
using muon::Work;

constexpr int kTable = 8;  // matrices of a launch
constexpr int kThreads = 256;
constexpr int kSumBlocks = 1024;  // workgroups of a matrix that take |u|, at most
constexpr float kScale = 4096.0f;
constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr int64_t kMaxElements = int64_t(1) << 28;  // of the padded matrix: its pairs stay below 2^30 bytes

struct Mat {
    float *P, *M;
    const void *G;
    int8_t *X, *XT, *A, *B;  // pairs: [mp][np], [np][mp], [mp][mp], [mp][mp]
    int8_t *XTn;             // where the next X^T goes: XT itself unless the product that reads it writes it too
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
    int first[kTable];  // of a launch's workgroups; INT_MAX past the last matrix
    int L;
};

struct Hyper {
    float mu, eps;
    double lr, wd;
    int nesterov;
    const float *lr_dev, *grad_scale;
    uint32_t *absmax;
};

// (without a loop whose every turn would wait for its load)
__device__ __forceinline__ int find(const Table &t, int id) {
    int l = 0;
#pragma unroll
    for (int i = 1; i < kTable; ++i) l += id >= t.first[i];
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
#pragma unroll 4
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

// ---- tiles of 32 F x 32 F, 16 threads a row ----------------------------------------
// A thread holds V = 2 F consecutive values of a row, so that a row's terms leave
// in whole 128-byte lines.

// V consecutive values of a row of pairs.
template <int V>
struct Few {
    typedef _Float16 type __attribute__((ext_vector_type(V)));
    type hi, lo;
    static __device__ __forceinline__ _Float16 *at(int8_t *base, int K, int r, int c) {
        return reinterpret_cast<_Float16 *>(base) + int64_t(r) * 2 * K + 2 * (c & ~31) + (c & 31);
    }
    __device__ __forceinline__ void load(int8_t *base, int K, int r, int c) {
        const _Float16 *p = at(base, K, r, c);
        hi = *reinterpret_cast<const type *>(p);
        lo = *reinterpret_cast<const type *>(p + 32);
    }
    static __device__ __forceinline__ void store(int8_t *base, int K, int r, int c, const float (&v)[V]) {
        type hi, lo;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            hi[e] = _Float16(v[e]);
            lo[e] = _Float16(v[e] - float(hi[e]));
        }
        _Float16 *p = at(base, K, r, c);
        *reinterpret_cast<type *>(p) = hi;
        *reinterpret_cast<type *>(p + 32) = lo;
    }
};

// A tile's transpose in LDS: the pitch spreads a column over the banks.
template <int F>
constexpr int kTurnPitch = 32 * F + (F == 1 ? 2 : 1);
template <int F>
constexpr int kTurn = 32 * F * kTurnPitch<F>;

template <int F>
__device__ __forceinline__ void turn_in(float *turned, int row, int c, const float (&v)[2 * F]) {
#pragma unroll
    for (int e = 0; e < 2 * F; ++e) turned[(c + e) * kTurnPitch<F> + row] = v[e];
}
template <int F>
__device__ __forceinline__ void turn_out(const float *turned, int row, int c, float (&v)[2 * F]) {
#pragma unroll
    for (int e = 0; e < 2 * F; ++e) v[e] = turned[row * kTurnPitch<F> + c + e];
}

// X = u / (|u| + eps) and X^T as pairs, zeros in the padding: a workgroup a tile
// of 64 x 64 of u (of P's layout).
template <class T>
__global__ __launch_bounds__(kThreads) void scale_kernel(Table t, Hyper h) {
    constexpr int F = 2, V = 2 * F, kRows = kThreads / 16, kPasses = 32 * F / kRows;
    __shared__ float turned[kTurn<F>];
    __shared__ double red[kThreads / 64];
    const int l = find(t, int(blockIdx.x));
    const Mat &a = t.mat[l];
    // rows and columns of P, and of its padded form
    const int rows = a.tall ? a.n : a.m, cols = a.cols, rp = a.tall ? a.np : a.mp, cp = a.tall ? a.mp : a.np;
    const int across = (cp + 63) / 64, b = int(blockIdx.x) - t.first[l];
    const int r0 = 64 * (b / across), c0 = 64 * (b % across), r = int(threadIdx.x) / 16, c = V * (int(threadIdx.x) % 16);
    const T *G = static_cast<const T *>(a.G);
    const float gs = h.grad_scale ? *h.grad_scale : 1.0f;
    float v[kPasses][V];
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int row = r0 + kRows * k + r, valid = row < rows ? cols - c0 - c : 0;
        const int64_t at = int64_t(row) * cols + c0 + c;
        const auto m = load_raw<float, V>(a.M + at, valid);
        const auto g = load_raw<T, V>(G + at, h.nesterov ? valid : 0);
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] = e < valid ? update_of(m[e], float(g[e]) * gs, h) : 0.0f;
    }
    double s = 0.0;
    for (int i = threadIdx.x; i < a.blocks; i += kThreads) s += a.sums[i];
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    s = (red[0] + red[1]) + (red[2] + red[3]);
    const double norm = sqrt(s) + double(h.eps);
    const double factor = norm > 0.0 ? double(kScale) / norm : (norm == 0.0 ? 0.0 : norm);  // (NaN stays one)
    int8_t *to = a.tall ? a.XT : a.X, *to_turned = a.tall ? a.X : a.XT;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int row = kRows * k + r;
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] = float(double(v[k][e]) * factor);
        turn_in<F>(turned, row, c, v[k]);
        if (r0 + row < rp && c0 + c < cp) Few<V>::store(to, cp, r0 + row, c0 + c, v[k]);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int row = kRows * k + r;
        turn_out<F>(turned, row, c, v[k]);
        if (c0 + row < cp && r0 + c < rp) Few<V>::store(to_turned, rp, c0 + row, r0 + c, v[k]);
    }
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
    w.S = w.K < 64 ? 1 : w.K / 64;
    // wide blocks, but places without a tile in the last one are a lane's idle workgroups
    // (36 tiles in blocks of 8: five of 1000 x 1000 798 us, in blocks of 4 694)
    w.width = 8;
    while (w.width > 1 && 32 * (-w.tiles & (w.width - 1)) > w.tiles) w.width /= 2;
    w.chunk = chunk;
    w.slots = (chunk + w.S - 1) / w.S + 1;
    w.lanes = int((int64_t(w.tiles + w.width - 1) / w.width * w.S + chunk - 1) / chunk);
    w.groups = (w.lanes + 7) / 8 * 8 * w.width;
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
    muon::pieces<256>(w, int(blockIdx.x), [&](int ti, int tj, int k0, int k1, float *to) {
        muon::piece256(w, ti, tj, k0, k1, to, sA0, sB0, sA1, sB1);
    });
}

// V values of P's row r from column c on; returns their largest magnitude's bits.
template <int V>
__device__ __forceinline__ uint32_t update(const Mat &a, float keep, float rate, int r, int c, const float (&x)[V]) {
    const int rows = a.tall ? a.n : a.m, valid = r < rows ? a.cols - c : 0;
    if (valid <= 0) return 0u;
    float *p = a.P + int64_t(r) * a.cols + c, o[V];
    const auto old = load_raw<float, V>(p, valid);
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        o[e] = old[e] * keep - x[e] * rate;
        if (e < valid) top = max(top, mag_bits(o[e]));
    }
    store_vec<float, V>(p, o, valid);
    return top;
}

// What follows a product, by NT threads: tile (r0, c0) of its sums (NSUM of them,
// in LDS as lay_small lays them) to the next operand (a symmetric one with the
// tile's mirror image, unless it is on the diagonal) or to P.
template <int F, int NT, int NSUM>
struct Finish {
    static constexpr int V = 2 * F, kRows = NT / 16, kPasses = 32 * F / kRows;
    static_assert(32 * F % kRows == 0, "whole passes");
    Few<V> own[kPasses];  // the block of A or X that goes into the polynomial, loaded ahead of the product

    __device__ __forceinline__ void load(const Mat &a, int product, int r0, int c0) {
        const int r = int(threadIdx.x) / 16, c = V * (int(threadIdx.x) % 16);
#pragma unroll
        for (int k = 0; k < kPasses; ++k) {
            if (product == AA) own[k].load(a.A, a.mp, r0 + kRows * k + r, c0 + c);
            if (product == BX) own[k].load(a.X, a.np, r0 + kRows * k + r, c0 + c);
        }
    }

    __device__ __forceinline__ void run(const Mat &a, const Hyper &h, int l, int product, bool mirror, bool last, int r0,
                                        int c0, const float *sums, float *turned) const {
        const int r = int(threadIdx.x) / 16, c = V * (int(threadIdx.x) % 16);
        const bool end = product == BX && last, turn = product == BX ? !end || a.tall : mirror;
        int8_t *to = product == XX ? a.A : product == AA ? a.B : a.X, *to_turned = product == BX ? a.XTn : to;
        const int K = product == BX ? a.np : a.mp;
        const double lr = h.lr_dev ? double(*h.lr_dev) : h.lr;
        const float keep = float(1.0 - lr * h.wd), rate = float(lr * double(a.scale) / double(kScale));
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kPasses; ++k) {
            const int row = kRows * k + r;
            float v[V];
            const float *p = sums + row * muon::kSmallPitch<F> + c;
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = p[e];
#pragma unroll
            for (int o = 1; o < NSUM; ++o)
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] += p[o * muon::kSmallTile<F> + e];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float x = float(own[k].hi[e]) + float(own[k].lo[e]);
                v[e] *= 1.0f / kScale;
                if (product == AA) v[e] = fmaf(kC, v[e], kB * x);
                if (product == BX) v[e] = fmaf(kA, x, v[e]);
            }
            if (turn) turn_in<F>(turned, row, c, v);
            if (!end) Few<V>::store(to, K, r0 + row, c0 + c, v);
            else if (!a.tall) top = max(top, update<V>(a, keep, rate, r0 + row, c0 + c, v));
        }
        if (turn) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kPasses; ++k) {
                const int row = kRows * k + r;
                float v[V];
                turn_out<F>(turned, row, c, v);
                if (!end) Few<V>::store(to_turned, a.mp, c0 + row, r0 + c, v);
                else top = max(top, update<V>(a, keep, rate, c0 + row, r0 + c, v));
            }
        }
        if (end && h.absmax) {
            top = wave_max_u32(top);
            if ((threadIdx.x & 63) == 0) publish_max_u32(h.absmax + l, top);
        }
    }
};

// The pieces of a product in tiles of 128 or 256 added up and finished: a
// workgroup 64 x 64 of a wavefront's share, a wavefront of it a block of 32 x 32.
template <int SIDE>
__global__ __launch_bounds__(kThreads) void finish_kernel(Table t, Hyper h, int product, int chunk, int last) {
    constexpr int F = SIDE / 64, kGroups = SIDE * SIDE / 4096, kAcross = F / 2;  // blocks of a wavefront's side; groups
    __shared__ float sums[muon::kSmallTile<2>];
    __shared__ float turned[kTurn<2>];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l = find(t, int(blockIdx.x));
    const Mat &a = t.mat[l];
    const Work w = work_of<SIDE>(a, product, chunk);
    const int id = int(blockIdx.x) - t.first[l], tile = id / kGroups, k = id % kGroups;
    const int part = k / (kAcross * kAcross), i = k % (kAcross * kAcross) / kAcross, j = k % kAcross;
    int ti, tj;
    muon::tile_at(w, SIDE, tile, ti, tj);
    const int r0 = SIDE * ti + (SIDE / 2) * (part >> 1) + 64 * i, c0 = SIDE * tj + (SIDE / 2) * (part & 1) + 64 * j;
    Finish<2, kThreads, 1> f;
    f.load(a, product, r0, c0);
    v4f v[4] = {};
    const int block = (part * F + 2 * i + (wave >> 1)) * F + 2 * j + (wave & 1);
    const int run = tile / w.width, q8 = tile - run * w.width;  // the tile's block and place in it
    const int first = run * w.S / chunk, end = ((run + 1) * w.S - 1) / chunk;
    for (int g = first; g <= end; ++g) {
        const int slot = run - g * chunk / w.S;
        const v4f *p = reinterpret_cast<const v4f *>(w.part + (int64_t(g * w.width + q8) * w.slots + slot) * (SIDE * SIDE)) +
                       block * 256 + lane;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += p[64 * q];
    }
    float *to = sums + (32 * (wave >> 1) + (lane & 31)) * muon::kSmallPitch<2> + 32 * (wave & 1) + 4 * (lane >> 5);
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<v4f *>(to + 8 * q) = v[q];
    __syncthreads();
    f.run(a, h, l, product, ti != tj, last, r0, c0, sums, turned);
}

// A product in small tiles, whole: tile 32 F a side, W wavefronts.  ALIKE: all
// matrices have the same sizes, and blockIdx.y is the matrix, so that what it needs
// is one trip to the arguments and not two (about 0.4 us of 4).
template <int F, int W, bool ALIKE>
__global__ __launch_bounds__(64 * W) void product_small_kernel(Table t, Hyper h, int product, int last) {
    constexpr int TS = 32 * F;
    static_assert((W * muon::kSmallTile<F> + kTurn<F>)*4 <= muon::kSmallLds<F, W>,
                  "the sums and a transpose fit where the stages were");
    __shared__ __attribute__((aligned(1024))) int8_t lds[muon::kSmallLds<F, W>];
    const int l = ALIKE ? int(blockIdx.y) : find(t, int(blockIdx.x));
    const Mat &a = t.mat[l];
    const Work w = work_of<TS>(a, product, 1);
    int ti, tj;
    muon::tile_at(w, TS, int(blockIdx.x) - (ALIKE ? 0 : t.first[l]), ti, tj);
    Finish<F, 64 * W, W> f;
    f.load(a, product, TS * ti, TS * tj);
    float *sums = reinterpret_cast<float *>(lds);
    {
        v16f acc[F][F];
        muon::sums_small<F, W>(w, ti, tj, lds, acc);
        __syncthreads();  // every wavefront has read its stages
        muon::lay_small<F>(acc, sums);
        __syncthreads();
    }
    f.run(a, h, l, product, ti != tj, last, TS * ti, TS * tj, sums, sums + W * muon::kSmallTile<F>);
}

// ---- host ------------------------------------------------------------------------

int64_t up(int64_t a, int64_t to) { return (a + to - 1) / to * to; }

// The side of the tiles that a batch's matrices are worked in, by the sum of m^2 n
// (a step's operations go with it) and the longest side; in us a step:
//   32 (of a whole reduction each): 256 x 256 69 against 106 in tiles of 64 and 215
//     in 128, 512 x 512 93 against 141; three of 512 x 512 (4.0e8) 157 and 141
//   64 (the same): 1024 x 1024 194 against 316 in tiles of 128, 1536 x 1536 (3.6e9)
//     522 and 527, four of 1000 x 1000 (4.0e9) 610 and 611
//   128 (the reduction cut into runs): 2048 x 2048 (8.6e9) 864 against 949 in tiles
//     of 256; with a long side also few operations, 128 x 32768 497 against 621
//     in tiles of 32 (128 x 8192: 298 and 208)
//   256, a matrix at a time: 2304 x 2304 (1.2e10) 1163 against 1156, 3000 x 3000
//     2110 against 2272, 4096 x 4096 4279 against 4823
constexpr double kLarge = 1.15e10;
double weight_of(const Mat &a) { return double(a.m) * a.m * a.n; }
int side_of(const Mat *mats, int L) {
    double sum = 0.0;
    int longest = 0;
    for (int l = 0; l < L; ++l) {
        sum += weight_of(mats[l]);
        if (mats[l].n > longest) longest = mats[l].n;
    }
    if (L == 1 && sum >= kLarge) return 256;
    return longest > 8192 || sum > 3.7e9 ? 128 : sum > 3.0e8 ? 64 : 32;
}

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
    Layout y{side_of(mats, L), {}, 0};
    const bool whole = y.side < 128;  // products and what follows them in one launch
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
        a.XTn = whole ? reinterpret_cast<int8_t *>(take(x)) : a.XT;
        a.A = reinterpret_cast<int8_t *>(take(s));
        a.B = reinterpret_cast<int8_t *>(take(s));
        a.sums = reinterpret_cast<double *>(take(kSumBlocks * sizeof(double)));
    }
    if (whole) return y;
    size_t most[kTable] = {};
    for (int p = 0; p < 3; ++p) {
        int64_t total = 0;
        const auto work = [&](int l, int chunk) {
            return y.side == 256 ? work_of<256>(mats[l], p, chunk) : work_of<128>(mats[l], p, chunk);
        };
        for (int l = 0; l < L; ++l) {
            const Work w = work(l, 1);
            total += int64_t(w.tiles + w.width - 1) / w.width * w.width * w.S;
        }
        y.chunk[p] = chunk_of(total, y.side == 256 ? 256 : 512);
        for (int l = 0; l < L; ++l) {
            const Work w = work(l, y.chunk[p]);
            const size_t b = size_t(w.lanes) * w.width * w.slots * y.side * y.side * sizeof(float);
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
    const int64_t b = (a.count + kThreads * 4 - 1) / (kThreads * 4);
    a.blocks = int(b < kSumBlocks ? b : kSumBlocks);
    return a;
}

bool size_ok(int64_t rows, int64_t cols) {
    return rows >= 1 && cols >= 1 && rows <= kMaxElements && cols <= kMaxElements &&
           up(rows, 256) * up(cols, 256) <= kMaxElements;
}

// Whether n floats at a and m at b have one in common.
bool overlap(const float *a, int64_t n, const float *b, int64_t m) { return a < b + m && b < a + n; }

// Takes the matrices from l on that share their launches; returns their number.
int take_batch(int L, const int64_t *rows, const int64_t *cols, int l, Mat *mats) {
    int k = 0;
    for (; k < kTable && l + k < L; ++k) {
        mats[k] = mat_of(rows[l + k], cols[l + k]);
        if (weight_of(mats[k]) >= kLarge) return k ? k : 1;
    }
    return k;
}

template <int F, int W>
void launch_small(Table &t, const Hyper &h, int p, bool last, hipStream_t st) {
    int groups = 0;
    for (int l = 0; l < t.L; ++l) {
        t.first[l] = groups;
        groups += work_of<32 * F>(t.mat[l], p, 1).tiles;
    }
    bool alike = true;
    for (int l = 1; l < t.L; ++l) alike = alike && t.mat[l].mp == t.mat[0].mp && t.mat[l].np == t.mat[0].np;
    if (alike)
        product_small_kernel<F, W, true>
            <<<dim3(unsigned(groups / t.L), unsigned(t.L)), dim3(64 * W), 0, st>>>(t, h, p, last);
    else
        product_small_kernel<F, W, false><<<dim3(unsigned(groups)), dim3(64 * W), 0, st>>>(t, h, p, last);
    for (int l = 0; p == BX && l < t.L; ++l) {
        int8_t *xt = t.mat[l].XT;
        t.mat[l].XT = t.mat[l].XTn;
        t.mat[l].XTn = xt;
    }
}

template <int SIDE>
void launch_product(Table &t, const Hyper &h, const Layout &y, int p, bool last, hipStream_t st) {
    int groups = 0;
    for (int l = 0; l < t.L; ++l) {
        t.first[l] = groups;
        groups += work_of<SIDE>(t.mat[l], p, y.chunk[p]).groups;
    }
    if (SIDE == 256) product256_kernel<<<dim3(unsigned(groups)), dim3(g256::NT), 0, st>>>(t.mat[0], p, y.chunk[p]);
    else product128_kernel<<<dim3(unsigned(groups)), dim3(kThreads), 0, st>>>(t, p, y.chunk[p]);
    constexpr int kGroups = SIDE * SIDE / 4096;  // workgroups of a tile
    groups = 0;
    for (int l = 0; l < t.L; ++l) {
        t.first[l] = groups;
        groups += work_of<SIDE>(t.mat[l], p, y.chunk[p]).tiles * kGroups;
    }
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
        Mat mats[kTable];
        const int k = take_batch(L, rows, cols, l, mats);
        const Layout y = lay_out(mats, k, nullptr);
        most = y.bytes > most ? y.bytes : most;
        l += k;
    }
    return most;
}

int ionn_muon_tile(int L, const int64_t *rows, const int64_t *cols, int l) {
    if (L < 1 || l < 0 || l >= L || ionn_muon_workspace_bytes(L, rows, cols) == 0) return -1;
    for (int first = 0;;) {
        Mat mats[kTable];
        const int k = take_batch(L, rows, cols, first, mats);
        if (l < first + k) return side_of(mats, k);
        first += k;
    }
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
    for (int l = 0; l < L; ++l) {  // (matrices are worked side by side)
        const int64_t n = rows[l] * cols[l];
        for (int k = 0; k < L; ++k) {
            const int64_t m = rows[k] * cols[k];
            const float *g = static_cast<const float *>(G[k]);
            const int64_t gm = (m * int64_t(dtype_size(g_dtype)) + 3) / 4;
            IONN_REQUIRE((k == l || (!overlap(P[l], n, P[k], m) && !overlap(M[l], n, M[k], m))) && !overlap(P[l], n, M[k], m),
                         IONN_ERR_ARG, "ionn_muon_step: matrix or momentum %d overlaps one of %d", l, k);
            IONN_REQUIRE(!overlap(P[l], n, g, gm) && !overlap(M[l], n, g, gm), IONN_ERR_ARG,
                         "ionn_muon_step: matrix or momentum %d overlaps gradient %d", l, k);
        }
    }
    const size_t need = ionn_muon_workspace_bytes(L, rows, cols);
    IONN_REQUIRE(workspace && aligned(workspace, 256) && workspace_bytes >= need, IONN_ERR_WORKSPACE,
                 "ionn_muon_step: needs a 256-byte aligned workspace of %zu bytes", need);
    hipStream_t st = as_stream(stream);
    for (int l = 0; l < L;) {
        Table t{};
        t.L = take_batch(L, rows, cols, l, t.mat);
        for (int i = t.L; i < kTable; ++i) t.first[i] = INT_MAX;
        for (int i = 0; i < t.L; ++i) {
            Mat &a = t.mat[i];
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
        with_dtype(g_dtype, [&](auto tag) {
            momentum_kernel<decltype(tag)><<<dim3(unsigned(blocks)), dim3(kThreads), 0, st>>>(t, h);
        });
        blocks = 0;
        for (int i = 0; i < t.L; ++i) {
            t.first[i] = blocks;
            blocks += ((t.mat[i].mp + 63) / 64) * ((t.mat[i].np + 63) / 64);
        }
        with_dtype(g_dtype, [&](auto tag) {
            scale_kernel<decltype(tag)><<<dim3(unsigned(blocks)), dim3(kThreads), 0, st>>>(t, h);
        });
        for (int k = 0; k < ns_steps; ++k)
            for (int p = 0; p < 3; ++p) {
                const bool last = p == BX && k + 1 == ns_steps;
                if (y.side == 32) launch_small<1, 8>(t, h, p, last, st);
                else if (y.side == 64) launch_small<2, 4>(t, h, p, last, st);
                else if (y.side == 256) launch_product<256>(t, h, y, p, last, st);
                else launch_product<128>(t, h, y, p, last, st);
            }
        if (int rc = check_launch("ionn_muon_step")) return rc;
        l += t.L;
    }
    return IONN_OK;
}

}  // extern "C"
