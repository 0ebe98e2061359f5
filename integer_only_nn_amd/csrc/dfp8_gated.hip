// The gated layer of a transformer's feed-forward block on DFP-8 operands (int8
// mantissas, one shared exponent per tensor), and its backward pass ("Mixed
// Precision Training of Convolutional Neural Networks using Integer
// Operations", sections 3 and 4: integer products, the operations around them
// in floating point).  W [2 H][IN] holds the gate's rows and then the up
// projection's, one tensor with one exponent.
//
//   (g | u) = fl(X W^T) 2^(eX + eW) + bias,  Y = act(g) u
//   dZ = (dY u act'(g) | dY act(g)) -> dZ8, edZ;  dX = fl(dZ8 W) 2^(edZ + eW),
//   G = fl(dZ8^T X) 2^(edZ + eX),  gb = column sums of dZ
//
// The forward product is a Linear layer's of 2 H outputs, in the same tiles and
// by the same rule (dfp8_plan.h), with one change: a tile's rows of W are half
// gate rows and half the up rows of the same outputs, so that both halves of an
// output meet in one workgroup's (or one lane's) sums and Y leaves in the
// epilogue.  The gradients' products are a Linear layer's of 2 H errors as they
// stand.
//
// Where larger tiles would be faster but for rows that are not whole 16-byte
// pieces, a product's operands are first copied into rows that are (in the
// workspace): 8192 x 4095 -> 4095, bfloat16, 266 us forward and 621 backward,
// straight in tiles of 64 743 and 1834; 2047 x 2047 -> 2047 33 and 78 against 53 and
// 139.
//
// The errors are two passes over dY, g and u, bound by HBM: one that takes the
// maximum and the column sums, one that rounds (the exponent needs the maximum
// of the whole tensor first, and a float32 copy of dZ would cost more bytes than
// computing it again).
//
// Measured: 8192 x 4096 -> 4096, bfloat16, silu: forward with z 265 us (2075 TOP/s;
// the library's int8 product reaches 2141), the errors' passes 53 and 52 us (205 and
// 273 MB), the two gradients' products 216 and 214; one row 7.9 us (W at 4.3 TB/s; 5.6
// where the XCDs' L2 hold most of it); 256 x 784 -> 256, float32, 3.5 forward and 4.8 +
// 4.7 + 5.2 backward.
#include <type_traits>

#include "dfp8_convert.h"
#include "dfp8_plan.h"

namespace ionn {
namespace {

using namespace dfp8;

constexpr int kThreads = 256;
constexpr int kRoundGroups = 2048;

// ---- forward -------------------------------------------------------------------

int64_t pitch_of(int64_t n) { return (n + 15) & ~int64_t(15); }
bool large(Path p) { return p == TILE256 || p == TILE128; }

// What copying operands of that many bytes takes, us.
double copy_us(int64_t bytes) { return 4.0 + double(bytes) / 5.0e6; }

// A Linear layer's plan for the 2 H rows of W; its tiles are counted in outputs.
// pitch: of the copies of X and W, 0 where they are taken as they are.
struct GatedPlan : Plan {
    int64_t pitch;
};
GatedPlan gated_plan(int64_t B, int64_t IN, int64_t H) {
    GatedPlan p{make_plan<true, true>(B, 2 * H, IN, true), 0};
    if (p.path == TILE && IN % 16) {
        const Plan c = make_plan<true, true>(B, 2 * H, IN, true, pitch_of(IN), pitch_of(IN));
        // (tiles of 64 take a fifth to a third longer than expected where rows are off
        // four bytes: 8192 x 1001 -> 2001 103 us against 63 with copies, 3000 x 1001 ->
        // 999 23 and 21; 2048 x 1000 -> 1020 13 and 17, 8192 x 1000 -> 2000 78 and 65)
        const double slow = IN % 4 ? 1.3 : 1.0;
        if (large(c.path) && c.us + copy_us((B + 2 * H) * pitch_of(IN)) < slow * p.us) p = GatedPlan{c, pitch_of(IN)};
    }
    if (p.path == ROWS) p.cols = 2;  // a group of gate rows and one of up rows
    p.tiles = ceil_div(B, 64) * ceil_div(H, 32);
    return p;
}

// A tensor's rows in a copy of another pitch (a multiple of 16, less than 16 above
// cols), zeros behind them.  cols >= 16, rows * pitch < 2^31.
struct Rows {
    const int8_t *from;
    int8_t *to;
    uint32_t cols, pitch, pieces;  // pieces of 16 bytes in all
};
struct Copies {
    Rows r[3];
    uint32_t first[3];  // workgroup
};
constexpr int kPiecesEach = 2;  // of a thread (8: 1000 x 1023 -> 2049 in tiles of 128 18.8 us against 18.0)

__global__ __launch_bounds__(kThreads) void copy_rows_kernel(Copies c) {
    typedef v4i loose __attribute__((aligned(1)));
    const int i = (blockIdx.x >= c.first[1]) + (blockIdx.x >= c.first[2]);
    const Rows &t = c.r[i];
    const uint32_t id0 = (blockIdx.x - c.first[i]) * (kThreads * kPiecesEach) + threadIdx.x, per = t.pitch / 16;
    v4i v[kPiecesEach];
    uint32_t past[kPiecesEach];
#pragma unroll
    for (int k = 0; k < kPiecesEach; ++k) {
        const uint32_t id = min(id0 + k * kThreads, t.pieces - 1), row = id / per, at = 16 * (id - row * per);
        const uint32_t from = min(at, t.cols - 16);  // the row's last 16 bytes, shifted
        past[k] = at - from;
        v[k] = *reinterpret_cast<const loose *>(t.from + uint64_t(row) * t.cols + from);
    }
#pragma unroll
    for (int k = 0; k < kPiecesEach; ++k) {
        const uint32_t id = id0 + k * kThreads;
        if (id < t.pieces) reinterpret_cast<v4i *>(t.to)[id] = shift_piece(v[k], int(past[k]));
    }
}

// Copies of tensors into rows of pitch_of(cols) bytes, one after the other.
struct Copier {
    Copies c{};
    int n = 0;
    uint32_t groups = 0;
    int8_t *to;
    explicit Copier(void *at) : to(static_cast<int8_t *>(at)) {}
    const int8_t *add(const int8_t *from, int64_t rows, int64_t cols) {
        const uint32_t pitch = uint32_t(pitch_of(cols)), pieces = uint32_t(rows * pitch / 16);
        c.r[n] = Rows{from, to, uint32_t(cols), pitch, pieces};
        c.first[n++] = groups;
        groups += uint32_t(ceil_div(pieces, kThreads * kPiecesEach));
        int8_t *p = to;
        to += rows * pitch;
        return p;
    }
    void launch(hipStream_t st) {
        for (int i = n; i < 3; ++i) c.first[i] = UINT32_MAX;
        if (groups) copy_rows_kernel<<<dim3(groups), dim3(kThreads), 0, st>>>(c);
    }
};

template <class T>
void launch_gated(const Plan &pl, Product p, hipStream_t st) {
    const Path path = path_of(pl, p.A, p.B);
    const dim3 block(NT);
    if (path == ROWS) {
        if (pl.rows == 1) launch_rows<T, 1, 2, true>(p, st);
        else if (pl.rows == 2) launch_rows<T, 2, 2, true>(p, st);
        else launch_rows<T, 4, 2, true>(p, st);
    } else if (path == TILE256) {
        tile256_kernel<T, true, true, false, true>
            <<<dim3(unsigned(ceil_div(p.M, 256) * ceil_div(p.N, 128))), dim3(g256::NT), 0, st>>>(
                p.A, p.lda, p.B, p.ldb, uint32_t(p.M * p.lda), uint32_t(2 * p.N * p.ldb), p.ep, p.M, p.N, p.K);
    } else if (path == TILE128) {
        tile128_kernel<T, true><<<dim3(unsigned(ceil_div(p.M, 128) * ceil_div(p.N, 64))), block, 0, st>>>(p);
    } else {
        const dim3 grid(unsigned(p.blocks));
        if (path == TINY) tile_kernel<T, 64, 64, 2, true, true, false, true, true><<<grid, block, 0, st>>>(p);
        else tile_kernel<T, 64, 64, 4, true, true, false, false, true><<<grid, block, 0, st>>>(p);
        if (p.split > 1) sum_gated_kernel<T><<<dim3(sum_groups(p)), block, 0, st>>>(p);
    }
}

// ---- the errors ----------------------------------------------------------------

// Two float32 values have a product of 48 bits, and rounding it to float32 on
// the way to 8 bits would now and then round a tie the wrong way: float32
// errors whose derivative is exact (none, relu) are taken in float64.  Products
// of 16-bit values are exact in float32.
template <class T, int ACT>
using Wide = std::conditional_t<sizeof(T) == 4 && (ACT == IONN_ACT_NONE || ACT == IONN_ACT_RELU), double, float>;

// An activation's value f and derivative df at z from one exponential.  With e =
// 2^x and p = 1 / (1 + e), 1 - p is e p: exact to its own size, where 1.0f - p is
// off by half a step of 1, which z (or, of gelu_tanh, z (1 + 0.13 z^2)) times it
// would carry into the result.  (p is 0 where e is infinite, and so is df.)
template <int ACT>
__device__ __forceinline__ void act_both(float z, float &f, float &df) {
    if (ACT == IONN_ACT_SILU || ACT == IONN_ACT_GELU_TANH) {
        const float x = ACT == IONN_ACT_SILU ? -kLog2e * z : z * fmaf(z * z, -kLog2e * kGeluK * kGeluC, -kLog2e * kGeluK);
        const float e = exp2_fast(x), p = __builtin_amdgcn_rcpf(1.0f + e), pq = p * (fminf(e, 0x1p126f) * p);
        const float y = within(z);
        f = above(z) * p;
        df = fmaf(ACT == IONN_ACT_SILU ? y : y * fmaf(y * y, 3.0f * kGeluK * kGeluC, kGeluK), pq, p);
    } else if (ACT == IONN_ACT_GELU) {
        const float x = fabsf(z), e = normal_exp(x), tail = normal_tail<kTermsGrad>(x, e);
        f = fmaf(-fminf(x, 30.0f), tail, fmaxf(z, 0.0f));
        df = fmaf(within(z) * kInvSqrt2Pi, e, z < 0.0f ? tail : 1.0f - tail);
    } else {
        f = act_value<ACT, kTermsGrad>(z);
        df = act_grad<ACT, kTermsGrad>(z);
    }
}

template <int ACT, class V>
__device__ __forceinline__ void gated_error(float dy, float g, float u, V &dg, V &du) {
    float f, df;
    act_both<ACT>(g, f, df);
    dg = V(dy) * V(u) * V(df);
    du = V(dy) * V(f);
}

__device__ __forceinline__ uint32_t mantissa_of(float x, int negE) { return dfp8_mantissa(x, negE); }
__device__ __forceinline__ uint32_t mantissa_of(double x, int negE) {
    const double y = fmin(fmax(ldexp(x, negE), -128.0), 127.0);
    return uint32_t(__double_as_longlong(y + 6755399441055744.0));  // 1.5 * 2^52
}

// Magnitude bits for the largest error's exponent.  Rounding a float64 product to
// float32 can take it to the next power of two ((1 + 2^-23) (2 - 2^-22) = 2 - 2^-45),
// so a value rounded up gives the bits below it, of its own power of two; what is
// beyond float32's numbers stays infinite.
__device__ __forceinline__ uint32_t top_bits(float x) { return mag_bits(x); }
__device__ __forceinline__ uint32_t top_bits(double x) {
    const float f = float(x);
    const uint32_t b = mag_bits(f);
    return b - uint32_t(b > 1u && b < 0x7f800000u && fabs(double(f)) > fabs(x));
}

__device__ __forceinline__ uint32_t block_max(uint32_t v) {
    __shared__ uint32_t red[kThreads / 64];
    v = wave_max_u32(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return max(max(red[0], red[1]), max(red[2], red[3]));
}

// The pieces (dy, g, u) of row r at columns c ..
template <class T, int VE>
struct Piece {
    typename Vec<T, VE>::type y, g, u;
    __device__ __forceinline__ void load(const T *dY, const T *Z, int64_t r, int H, int c, int valid) {
        y = load_raw<T, VE>(dY + r * H + c, valid);
        g = load_raw<T, VE>(Z + 2 * r * H + c, valid);
        u = load_raw<T, VE>(Z + 2 * r * H + H + c, valid);
    }
};

// Workgroup (strip, chunk): the strip's columns over the chunk's rows, four
// wavefronts of 64 / lanes rows each at a time (act_layout of the H columns).
template <class T, int ACT>
__global__ __launch_bounds__(kThreads) void gated_sums_kernel(const T *__restrict__ dY, const T *__restrict__ Z,
                                                              int64_t B, int H, int lanes_log, int64_t chunk_rows,
                                                              uint32_t *__restrict__ part_max,
                                                              float *__restrict__ part_sum) {
    constexpr int VE = 16 / sizeof(T);
    __shared__ float fold[kThreads / 64][2][64 * VE];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lanes = 1 << lanes_log, per_wave = 64 >> lanes_log;
    const int c = (int(blockIdx.x) * lanes + (lane & (lanes - 1))) * VE;
    const int64_t r1 = min(B, int64_t(blockIdx.y + 1) * chunk_rows);
    float s[2][VE] = {};
    uint32_t m = 0;
    if (c < H) {
        const int valid = H - c, step = (kThreads / 64) * per_wave;
        auto add = [&](const Piece<T, VE> &p) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                Wide<T, ACT> dg, du;
                gated_error<ACT>(float(p.y[e]), float(p.g[e]), float(p.u[e]), dg, du);
                s[0][e] += float(dg);
                s[1][e] += float(du);
                // (past a row's end all three are 0, and so are both errors)
                m = max(m, max(top_bits(dg), top_bits(du)));
            }
        };
        int64_t r = int64_t(blockIdx.y) * chunk_rows + wave * per_wave + (lane >> lanes_log);
        for (; r + step < r1; r += 2 * step) {  // two rows' loads in flight
            Piece<T, VE> p[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) p[k].load(dY, Z, r + k * step, H, c, valid);
#pragma unroll
            for (int k = 0; k < 2; ++k) add(p[k]);
        }
        for (; r < r1; r += step) {
            Piece<T, VE> p;
            p.load(dY, Z, r, H, c, valid);
            add(p);
        }
    }
    // the row groups of a wavefront, then the wavefronts
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            for (int off = lanes; off < 64; off <<= 1) s[k][e] += __shfl_xor(s[k][e], off, 64);
            fold[wave][k][(lane & (lanes - 1)) * VE + e] = s[k][e];
        }
    m = block_max(m);  // (its barrier orders fold as well)
    if (threadIdx.x == 0) part_max[blockIdx.y * gridDim.x + blockIdx.x] = m;
    if (part_sum == nullptr) return;
    for (int i = threadIdx.x; i < 2 * lanes * VE; i += kThreads) {
        const int k = i >= lanes * VE, j = i - k * lanes * VE, col = int(blockIdx.x) * lanes * VE + j;
        if (col < H)
            part_sum[(2 * int64_t(blockIdx.y) + k) * H + col] =
                (fold[0][k][j] + fold[1][k][j]) + (fold[2][k][j] + fold[3][k][j]);
    }
}

// Workgroups below n_round round the errors, each every n_round-th (strip, chunk)
// as above (each reads all maxima, so there are at most kRoundGroups); those from it
// on add up the chunks' column sums, 64 columns at a time, every fourth chunk
// per wavefront.
template <class T, int ACT>
__global__ __launch_bounds__(kThreads) void gated_round_kernel(
    const T *__restrict__ dY, const T *__restrict__ Z, int64_t B, int H, int lanes_log, int strips, int64_t chunk_rows,
    int n_round, const uint32_t *__restrict__ part_max, int nparts, const float *__restrict__ part_sum, int chunks,
    int8_t *__restrict__ dZ8, int32_t *__restrict__ edZ, float *__restrict__ gb, int32_t *__restrict__ status) {
    constexpr int VE = 16 / sizeof(T);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (int(blockIdx.x) >= n_round) {
        __shared__ float red[kThreads / 64][64];
        const int64_t cols = 2 * int64_t(H), step = (int64_t(gridDim.x) - n_round) * 64;
        for (int64_t c0 = int64_t(int(blockIdx.x) - n_round) * 64; c0 < cols; c0 += step) {
            const int64_t c = c0 + lane;
            float s = 0.0f;
            if (c < cols) {
#pragma unroll 8
                for (int k = wave; k < chunks; k += kThreads / 64) s += part_sum[int64_t(k) * cols + c];
            }
            red[wave][lane] = s;
            __syncthreads();
            if (wave == 0 && c < cols) gb[c] = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
            __syncthreads();
        }
        return;
    }
    uint32_t m = 0;
    for (int i = threadIdx.x; i < nparts; i += kThreads) m = max(m, part_max[i]);
    m = block_max(m);
    const int E = dfp8_exponent(m);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *edZ = E;
        if (status) *status = dfp8_status(m, E);
    }
    const int lanes = 1 << lanes_log, per_wave = 64 >> lanes_log, step = (kThreads / 64) * per_wave;
    auto put = [&](const Piece<T, VE> &p, int64_t r, int c, int valid) __attribute__((always_inline)) {
        uint32_t qg[VE], qu[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            Wide<T, ACT> dg, du;
            gated_error<ACT>(float(p.y[e]), float(p.g[e]), float(p.u[e]), dg, du);
            qg[e] = mantissa_of(dg, -E);
            qu[e] = mantissa_of(du, -E);
        }
        int8_t *z = dZ8 + 2 * r * H + c;
        store_bytes(z, qg, VE, valid);
        store_bytes(z + H, qu, VE, valid);
    };
    for (int unit = int(blockIdx.x); unit < nparts; unit += n_round) {
        const int chunk = unit / strips, c = ((unit - chunk * strips) * lanes + (lane & (lanes - 1))) * VE, valid = H - c;
        if (valid <= 0) continue;
        const int64_t r1 = min(B, int64_t(chunk + 1) * chunk_rows);
        int64_t r = int64_t(chunk) * chunk_rows + wave * per_wave + (lane >> lanes_log);
        for (; r + step < r1; r += 2 * step) {  // two rows' loads in flight
            Piece<T, VE> p[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) p[k].load(dY, Z, r + k * step, H, c, valid);
#pragma unroll
            for (int k = 0; k < 2; ++k) put(p[k], r + k * step, c, valid);
        }
        for (; r < r1; r += step) {
            Piece<T, VE> p;
            p.load(dY, Z, r, H, c, valid);
            put(p, r, c, valid);
        }
    }
}

// Bytes of the maxima and of the column sums' partial rows.
size_t error_bytes(int64_t B, int64_t H) {
    size_t most = 0;
    for (size_t es : {size_t(2), size_t(4)}) {
        const ActLayout a = act_layout(B, H, es);
        const size_t maxima = (size_t(a.strips) * a.chunks * sizeof(uint32_t) + 15) & ~size_t(15);
        const size_t b = maxima + size_t(a.chunks) * 2 * H * sizeof(float);
        most = b > most ? b : most;
    }
    return (most + 15) & ~size_t(15);
}

void launch_errors(const void *dY, const void *Z, int act, int dtype, int64_t B, int64_t H, int8_t *dZ8, int32_t *edZ,
                   float *gb, int32_t *status, void *workspace, hipStream_t st) {
    const ActLayout a = act_layout(B, H, dtype_size(dtype));
    const int nparts = a.strips * a.chunks, n_round = nparts < kRoundGroups ? nparts : kRoundGroups;
    uint32_t *maxima = static_cast<uint32_t *>(workspace);
    float *sums = gb ? reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                                 ((size_t(nparts) * sizeof(uint32_t) + 15) & ~size_t(15)))
                     : nullptr;
    int lanes_log = 0;
    while ((1 << lanes_log) < a.lanes) ++lanes_log;
    // (at most 2^20 workgroups of sums: one for each 64 of 2^30 columns and the others would be too many threads)
    const unsigned n_sum = gb ? unsigned(2 * H <= int64_t(64) << 20 ? (2 * H + 63) / 64 : int64_t(1) << 20) : 0u;
    with_dtype(dtype, [&](auto tag) {
        using T = decltype(tag);
        const T *y = static_cast<const T *>(dY), *z = static_cast<const T *>(Z);
        with_act(act, [&](auto ac) {
            constexpr int ACT = decltype(ac)::value;
            gated_sums_kernel<T, ACT><<<dim3(unsigned(a.strips), unsigned(a.chunks)), dim3(kThreads), 0, st>>>(
                y, z, B, int(H), lanes_log, a.rows, maxima, sums);
            gated_round_kernel<T, ACT><<<dim3(unsigned(n_round) + n_sum), dim3(kThreads), 0, st>>>(
                y, z, B, int(H), lanes_log, a.strips, a.rows, n_round, maxima, nparts, sums, a.chunks, dZ8, edZ, gb,
                status);
        });
    });
}

// The gradients' products and which of their operands are copied.
struct BackwardPlan {
    BackwardSizes s;
    bool copy_Z, copy_X, copy_W;
    size_t copy_bytes() const {
        return (copy_Z ? size_t(s.B) * s.ldz : 0) + (copy_X ? size_t(s.B) * s.ldx : 0) + (copy_W ? size_t(s.OUT) * s.ldw : 0);
    }
};
BackwardPlan backward_plan(int64_t B, int64_t IN, int64_t H) {
    const int64_t OUT = 2 * H;
    BackwardPlan p{{B, IN, OUT, OUT, IN, IN}, false, false, false};
    const bool z = OUT % 16 != 0, in = IN % 16 != 0;
    if (!z && !in) return p;
    Plan d, g, dc, gc;
    backward_plans(p.s, d, g);
    backward_plans({B, IN, OUT, pitch_of(OUT), pitch_of(IN), pitch_of(IN)}, dc, gc);
    const int64_t bz = z ? B * pitch_of(OUT) : 0, bx = in ? B * pitch_of(IN) : 0, bw = in ? OUT * pitch_of(IN) : 0;
    bool for_d = d.path == TILE && large(dc.path), for_g = g.path == TILE && large(gc.path);
    // (with copies for both: 1025 x 4095 -> 1001 55 us against 78, 2000 x 3001 -> 501 55
    // and 68; for one alone there is less to gain: 300 x 4095 -> 8192 152 without, 159
    // with, 1024 x 2050 -> 2050 80 and 88)
    const double slow = IN % 4 || OUT % 4 ? 1.15 : 1.0;
    if (!(for_d && for_g && dc.us + gc.us + copy_us(bz + bx + bw) < slow * (d.us + g.us))) {
        for_d = for_d && dc.us + copy_us(bz + bw) < d.us;
        for_g = for_g && gc.us + copy_us(bz + bx) < g.us;
    }
    p.copy_Z = z && (for_d || for_g);
    p.copy_X = in && for_g;
    p.copy_W = in && for_d;
    if (p.copy_Z) p.s.ldz = pitch_of(OUT);
    if (p.copy_X) p.s.ldx = pitch_of(IN);
    if (p.copy_W) p.s.ldw = pitch_of(IN);
    return p;
}

bool gated_sizes_ok(int64_t B, int64_t IN, int64_t H) {
    return H >= 0 && H <= kMaxSide / 2 && sizes_ok(B, IN, 2 * H) && tiles_ok(B, 2 * H);
}

bool apart(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return !a || !b || x + na <= y || y + nb <= x;
}

}  // namespace
}  // namespace ionn

using namespace ionn;
using namespace ionn::dfp8;

extern "C" {

size_t dfp8_gated_fwd_workspace_bytes(int64_t B, int64_t IN, int64_t H) {
    if (!gated_sizes_ok(B, IN, H) || B == 0 || H == 0) return 0;
    const GatedPlan p = gated_plan(B, IN, H);
    return p.pitch ? size_t(B + 2 * H) * p.pitch : part_bytes(p, B, 2 * H);
}

int dfp8_gated_fwd(const int8_t *X, const int32_t *eX, const int8_t *W, const int32_t *eW, const float *bias, int act,
                   void *Z, void *Y, int dtype, int64_t B, int64_t IN, int64_t H, uint32_t *absmax_Y, void *workspace,
                   size_t workspace_bytes, void *stream) {
    clear_error();
    IONN_REQUIRE(dtype_ok(dtype), IONN_ERR_ARG, "dfp8_gated_fwd: dtype = %d", dtype);
    IONN_REQUIRE(act >= IONN_ACT_NONE && act <= IONN_ACT_SILU, IONN_ERR_ARG, "dfp8_gated_fwd: act = %d", act);
    IONN_REQUIRE(gated_sizes_ok(B, IN, H) && IN <= IONN_DFP8_MAX_REDUCTION, IONN_ERR_SHAPE,
                 "dfp8_gated_fwd: B=%lld IN=%lld H=%lld (IN at most %d)", (long long)B, (long long)IN, (long long)H,
                 IONN_DFP8_MAX_REDUCTION);
    if (B == 0 || H == 0) return IONN_OK;
    IONN_REQUIRE(Y && eX && eW && (IN == 0 || (X && W)), IONN_ERR_ARG, "dfp8_gated_fwd: NULL tensor");
    const size_t es = dtype_size(dtype), out = size_t(B) * H * es;
    IONN_REQUIRE(apart(Y, out, Z, 2 * out), IONN_ERR_ARG, "dfp8_gated_fwd: Z must not overlap Y");
    IONN_REQUIRE(aligned(Y, es) && aligned(Z, es) && aligned(bias, 4) && aligned(eX, 4) && aligned(eW, 4) &&
                     aligned(absmax_Y, 4),
                 IONN_ERR_ALIGN, "dfp8_gated_fwd: tensors must be aligned to their element size");
    const size_t need = dfp8_gated_fwd_workspace_bytes(B, IN, H);
    IONN_REQUIRE(need == 0 || (workspace && aligned(workspace, 16) && workspace_bytes >= need), IONN_ERR_WORKSPACE,
                 "dfp8_gated_fwd: needs a 16-byte aligned workspace of %zu bytes", need);
    const Epi ep{eX, eW, bias, nullptr, Z, Y, absmax_Y, act};
    const GatedPlan plan = gated_plan(B, IN, H);
    Product p = make_product(plan, X, IN, W, IN, ep, B, H, IN, workspace);
    Copier copies(workspace);
    if (plan.pitch) {
        p.A = copies.add(X, B, IN);
        p.B = copies.add(W, 2 * H, IN);
        p.lda = p.ldb = plan.pitch;
    }
    Product both = p;  // its tiles are those of the 2 H rows of W
    both.N = int(2 * H);
    IONN_REQUIRE(launches(plan, both), IONN_ERR_SHAPE, "dfp8_gated_fwd: B=%lld H=%lld have too many tiles", (long long)B,
                 (long long)H);
    copies.launch(as_stream(stream));
    with_dtype(dtype, [&](auto tag) { launch_gated<decltype(tag)>(plan, p, as_stream(stream)); });
    return check_launch("dfp8_gated_fwd");
}

size_t dfp8_gated_bwd_workspace_bytes(int64_t B, int64_t IN, int64_t H) {
    if (!gated_sizes_ok(B, IN, H) || B == 0 || H == 0) return 0;
    const BackwardPlan p = backward_plan(B, IN, H);
    return error_bytes(B, H) + (IN > 0 ? backward_part_bytes(p.s) + p.copy_bytes() : 0);
}

int dfp8_gated_bwd(const void *dY, const void *Z, int act, int dtype, const int8_t *X, const int32_t *eX,
                   const int8_t *W, const int32_t *eW, int8_t *dZ8, int32_t *edZ, void *dX, void *G, float *gb,
                   int64_t B, int64_t IN, int64_t H, int32_t *status_out, void *workspace, size_t workspace_bytes,
                   void *stream) {
    clear_error();
    IONN_REQUIRE(dtype_ok(dtype), IONN_ERR_ARG, "dfp8_gated_bwd: dtype = %d", dtype);
    IONN_REQUIRE(act >= IONN_ACT_NONE && act <= IONN_ACT_SILU, IONN_ERR_ARG, "dfp8_gated_bwd: act = %d", act);
    IONN_REQUIRE(gated_sizes_ok(B, IN, H) && (dX == nullptr || 2 * H <= IONN_DFP8_MAX_REDUCTION) &&
                     (G == nullptr || B <= IONN_DFP8_MAX_REDUCTION) && tiles_ok(B, IN) && tiles_ok(2 * H, IN),
                 IONN_ERR_SHAPE, "dfp8_gated_bwd: B=%lld IN=%lld H=%lld (2 H with dX, B with G: at most %d)",
                 (long long)B, (long long)IN, (long long)H, IONN_DFP8_MAX_REDUCTION);
    const bool error = B > 0 && H > 0;  // there is an error to go by
    IONN_REQUIRE(edZ && (!error || (dY && Z && dZ8)), IONN_ERR_ARG, "dfp8_gated_bwd: NULL dY, Z, dZ8 or edZ");
    IONN_REQUIRE(!error || IN == 0 || ((dX == nullptr || (W && eW)) && (G == nullptr || (X && eX))), IONN_ERR_ARG,
                 "dfp8_gated_bwd: dX needs W and eW, G needs X and eX");
    const size_t es = dtype_size(dtype);
    IONN_REQUIRE(aligned(dY, es) && aligned(Z, es) && aligned(dX, es) && aligned(G, es) && aligned(gb, 4) &&
                     aligned(eX, 4) && aligned(eW, 4) && aligned(edZ, 4) && aligned(status_out, 4),
                 IONN_ERR_ALIGN, "dfp8_gated_bwd: tensors must be aligned to their element size");
    const size_t need = dfp8_gated_bwd_workspace_bytes(B, IN, H);
    IONN_REQUIRE(need == 0 || (workspace && aligned(workspace, 16) && workspace_bytes >= need), IONN_ERR_WORKSPACE,
                 "dfp8_gated_bwd: needs a 16-byte aligned workspace of %zu bytes", need);
    hipStream_t st = as_stream(stream);
    if (!error) {
        zero_bytes(edZ, 4, st);
        zero_bytes(status_out, 4, st);
        zero_bytes(dX, B * IN * int64_t(es), st);
        zero_bytes(G, 2 * H * IN * int64_t(es), st);
        zero_bytes(gb, 8 * H, st);
        return check_launch("dfp8_gated_bwd");
    }
    const BackwardPlan plan = backward_plan(B, IN, H);
    char *parts = static_cast<char *>(workspace) + error_bytes(B, H);
    BackwardProducts p{dZ8, X, W, edZ, eX, eW, dX, G, plan.s, parts};
    Copier copies(parts + (IN > 0 ? backward_part_bytes(plan.s) : 0));
    if (plan.copy_Z && (dX || G)) p.dZ8 = copies.add(dZ8, B, 2 * H);
    if (plan.copy_X && G) p.X = copies.add(X, B, IN);
    if (plan.copy_W && dX) p.W = copies.add(W, 2 * H, IN);
    IONN_REQUIRE(IN == 0 || backward_launches(p), IONN_ERR_SHAPE,
                 "dfp8_gated_bwd: B=%lld IN=%lld H=%lld have too many tiles", (long long)B, (long long)IN, (long long)H);
    launch_errors(dY, Z, act, dtype, B, H, dZ8, edZ, gb, status_out, workspace, st);
    if (int rc = check_launch("dfp8_gated_bwd")) return rc;
    if (IN == 0) return IONN_OK;
    copies.launch(st);
    launch_backward_products(p, dtype, st);
    return check_launch("dfp8_gated_bwd");
}

}  // extern "C"
