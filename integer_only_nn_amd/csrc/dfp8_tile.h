// Tiled int8 product with a floating epilogue, for any sizes, row lengths and
// addresses (gfx950, v_mfma_i32_32x32x32_i8).
//
// s[m][n] = sum_k A(m, k) B(n, k), exact in int32.  Each operand is K-major
// (element (r, k) at base[r * ld + k]) or M-major (base[k * ld + r]), as in
// the three products of a Linear layer:
//   fwd   A = X   [B][IN],  B = W [OUT][IN]   (both K-major)
//   dgrad A = dZ8 [B][OUT], B = W [OUT][IN]   (K-major, M-major)
//   wgrad A = dZ8 [B][OUT], B = X [B][IN]     (both M-major)
//
// A workgroup of four wavefronts (2 x 2) takes a BM x BN tile in 128-deep K
// steps, double-buffered in LDS.  A step's arithmetic is far shorter than a
// trip to memory, so DEPTH steps of 16-byte pieces are in flight in registers.
// Their loads are unconditional (a lane-dependent branch around a load makes
// the compiler wait for everything in flight) and in bounds: a piece that a
// row's or the tensor's end cuts is loaded so that it ends there and shifted
// down on its way to LDS, a row or k past the end repeats the last one, and
// A's values past K become 0.  Pieces start at whatever byte they start on,
// so odd sizes cost a shift in the last piece and no byte-wise path.
//
// Bound by the trip to memory where there are few steps (256 x 784 x 256: 5.4 us,
// 3.3 of them a launch in a graph; 512^3 4.3 us) and by the 64 bytes a clock
// that a compute unit loads where there are many tiles (1000 x 1024 x 2048 8.4
// us; pieces off their 16 bytes and a last column of tiles for one output,
// 1000 x 1023 x 2049, 15.6 us).  128 x 128 tiles (dfp8_tile128.h) halve those bytes
// but leave half the compute units without work at these sizes: 11.2 us.
//
// LDS layouts, without bank conflicts in either direction:
//   K-major [rows][128 B]: 16-byte piece c of row r at position c ^ fK(r & 15)
//     (gemm256.h); a fragment is one 16-byte read.
//   M-major [128 k][R B]: piece c of row k at position c ^ fT(k), fT(k) =
//     2 ((k >> 1) & 3) for R = 128 (two rows fill the 256-byte bank window)
//     and 2 ((k >> 2) & 1) for R = 64 (four rows do); a fragment is two
//     ds_read_b64_tr_b8, which return eight k of one row each.
#pragma once

#include "float_ops.h"
#include "gemm256.h"

namespace ionn {
namespace dfp8 {

typedef int v2i __attribute__((ext_vector_type(2)));

constexpr int BK = 128, NT = 256;

// LDS operations of a wavefront take effect in program order; this keeps the
// compiler to it where lanes exchange values.
__device__ __forceinline__ void in_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The epilogue of a product.  z = fl(s) 2^(ea + eb) (+ bias), y = act(z) (+
// residual): outputs of type T at row pitch N (rows are contiguous).
struct Epi {
    const int32_t *ea, *eb;
    const float *bias;     // nullable
    const void *residual;  // nullable, may be y
    void *z;               // nullable
    void *y;
    uint32_t *absmax;      // nullable
    int act;
};

// 16 bytes at base + off of which the first `valid` are wanted (the others
// come back as zeros); bytes [0, off + valid) of the tensor exist.
__device__ __forceinline__ v4i load_piece(const int8_t *base, int64_t off, int valid) {
    typedef v4i loose __attribute__((aligned(1)));
    if (valid >= 16) return *reinterpret_cast<const loose *>(base + off);
    v4i v = {0, 0, 0, 0};
    if (valid <= 0) return v;
    const int sh = 16 - valid;
    if (off >= sh) {
        const v4i w = *reinterpret_cast<const loose *>(base + off - sh);
        uint64_t lo = uint32_t(w.x) | uint64_t(uint32_t(w.y)) << 32, hi = uint32_t(w.z) | uint64_t(uint32_t(w.w)) << 32;
        if (sh >= 8) {
            lo = hi;
            hi = 0;
        }
        const int b = 8 * (sh & 7);
        if (b) {
            lo = lo >> b | hi << (64 - b);
            hi >>= b;
        }
        v = v4i{int(lo), int(lo >> 32), int(hi), int(hi >> 32)};
    } else {  // the first bytes of the tensor
        uint32_t w[4] = {0, 0, 0, 0};
        for (int i = 0; i < valid; ++i) w[i >> 2] |= uint32_t(uint8_t(base[off + i])) << (8 * (i & 3));
        v = v4i{int(w[0]), int(w[1]), int(w[2]), int(w[3])};
    }
    return v;
}

// v shifted down by sh bytes (zeros from above), sh >= 0.
__device__ __forceinline__ v4i shift_piece(const v4i &v, int sh) {
    uint32_t w[5] = {uint32_t(v.x), uint32_t(v.y), uint32_t(v.z), uint32_t(v.w), 0u};
    if (sh & 8) {
        w[0] = w[2];
        w[1] = w[3];
        w[2] = w[3] = 0u;
    }
    if (sh & 4) {
        w[0] = w[1];
        w[1] = w[2];
        w[2] = w[3];
        w[3] = 0u;
    }
    v4i o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = sh >= 16 ? 0 : int(__builtin_amdgcn_alignbyte(w[i + 1], w[i], uint32_t(sh & 3)));
    return o;
}

template <int R>
__device__ __forceinline__ int fT(int k) {
    return R == 128 ? 2 * ((k >> 1) & 3) : 2 * ((k >> 2) & 1);
}

// One operand's tile of R rows: a step's pieces to registers, then to LDS.
// TINY: the contiguous side is shorter than a piece.
// HALF: a gated layer's weights [2 rows][kdim]; the tile's first R / 2 rows are
// gate rows from r0 / 2 on, the others the up rows of the same outputs.
template <int R, bool KMAJOR, bool TINY, bool HALF = false>
struct Stage {
    static_assert(!HALF || KMAJOR, "the gated layer's weights are K-major");
    static constexpr int kPer = R * BK / 16 / NT;
    static_assert(R * BK / 16 % NT == 0, "whole pieces per thread");
    v4i reg[kPer];
    __device__ __forceinline__ void load(const int8_t *base, int64_t ld, int rows, int kdim, int r0, int k0) {
        typedef v4i loose __attribute__((aligned(1)));
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int id = j * NT + int(threadIdx.x);
            const int r = r0 + (KMAJOR ? id / (BK / 16) : 16 * (id % (R / 16)));
            const int k = k0 + (KMAJOR ? 16 * (id % (BK / 16)) : id / (R / 16));
            if (HALF) {
                const int t = id / (BK / 16), h = t >= R / 2;
                const int64_t row = int64_t(h) * rows + min(r0 / 2 + t - h * (R / 2), rows - 1);
                reg[j] = TINY ? load_piece(base, row * ld + k, kdim - k)
                              : *reinterpret_cast<const loose *>(base + row * ld + min(k, kdim - 16));
            } else if (TINY && KMAJOR)
                reg[j] = load_piece(base, r * ld + k, r < rows ? kdim - k : 0);
            else if (TINY)
                reg[j] = load_piece(base, k * ld + r, k < kdim ? rows - r : 0);
            else if (KMAJOR)
                reg[j] = *reinterpret_cast<const loose *>(base + min(r, rows - 1) * ld + min(k, kdim - 16));
            else
                reg[j] = *reinterpret_cast<const loose *>(base + min(k, kdim - 1) * ld + min(r, rows - 16));
        }
    }
    // r0, k0: of the step in the registers
    __device__ __forceinline__ void store(int8_t *lds, int rows, int kdim, int r0, int k0) {
        if (!TINY && (k0 + BK > kdim || (!KMAJOR && r0 + R > rows))) {  // a step or a tile that an end cuts
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int id = j * NT + int(threadIdx.x);
                if (KMAJOR) {
                    reg[j] = shift_piece(reg[j], max(0, k0 + 16 * (id % (BK / 16)) - (kdim - 16)));
                } else {
                    const bool past = k0 + id / (R / 16) >= kdim;
                    reg[j] = shift_piece(reg[j], past ? 16 : max(0, r0 + 16 * (id % (R / 16)) - (rows - 16)));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int id = j * NT + int(threadIdx.x);
            int o;
            if (KMAJOR) {
                const int r = id / (BK / 16), c = id % (BK / 16);
                o = r * BK + 16 * (c ^ g256::fK(r & 15));
            } else {
                const int k = id / (R / 16), c = id % (R / 16);
                o = k * R + 16 * (c ^ fT<R>(k));
            }
            *reinterpret_cast<v4i *>(lds + o) = reg[j];
        }
    }
};

// The fragment of rows rw .. rw + 31 (lane: row lane % 32) and k = 32 sl + 16
// (lane / 32) .. + 15 of the tile.
template <int R, bool KMAJOR>
__device__ __forceinline__ v4i read_frag(const int8_t *lds, int rw, int sl, int lane) {
    if (KMAJOR) {
        const int r = rw + (lane & 31), c = 2 * sl + (lane >> 5);
        return *reinterpret_cast<const v4i *>(lds + r * BK + 16 * (c ^ g256::fK(r & 15)));
    }
    typedef __attribute__((address_space(3))) v2i lds_v2i;
    const int g = lane >> 4, i = lane & 15;
    const int c = (rw >> 4) + (g & 1);
    v4i out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int k = 32 * sl + 16 * (g >> 1) + 8 * h + (i >> 1);
        const int8_t *p = lds + k * R + 16 * (c ^ fT<R>(k)) + 8 * (i & 1);
        const v2i v = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)(p));
        out[2 * h] = v.x;
        out[2 * h + 1] = v.y;
    }
    return out;
}

// The bias of columns n .. n + V - 1 (zeros without one, or past N).
template <int V>
__device__ __forceinline__ void load_bias(const Epi &ep, int n, int N, float (&b)[V]) {
    const auto raw = load_raw<float, V>(ep.bias + n, ep.bias ? N - n : 0);
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = raw[i];
}

// The same for the two halves of a gated layer's bias [2 H]: columns n .. of each.
template <int V>
__device__ __forceinline__ void load_bias2(const Epi &ep, int n, int H, float (&bg)[V], float (&bu)[V]) {
    load_bias(ep, n, H, bg);
    const auto raw = load_raw<float, V>(ep.bias + H + n, ep.bias ? H - n : 0);
#pragma unroll
    for (int i = 0; i < V; ++i) bu[i] = raw[i];
}

// A gated layer's outputs n .. n + V - 1 of row m from the sums of its gate and
// up halves: y = act(g) u at row pitch H, z = (g, u) at 2 H.
template <class T, int ACT, int V>
__device__ __forceinline__ uint32_t finish_gated(const int (&sg)[V], const int (&su)[V], const Epi &ep, int e2,
                                                 const float (&bg)[V], const float (&bu)[V], int64_t m, int n, int M,
                                                 int H) {
    if (m >= M || n >= H) return 0u;
    const int valid = H - n;
    float g[V], u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        g[i] = __builtin_amdgcn_ldexpf(float(sg[i]), e2) + bg[i];
        u[i] = __builtin_amdgcn_ldexpf(float(su[i]), e2) + bu[i];
    }
    if (ep.z) {
        T *z = static_cast<T *>(ep.z) + 2 * m * H + n;
        store_vec<T, V>(z, g, valid);
        store_vec<T, V>(z + H, u, valid);
    }
    float o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = act_value<ACT, kTermsValue<T>>(g[i]) * u[i];
    store_vec<T, V>(static_cast<T *>(ep.y) + m * H + n, o, valid);
    uint32_t top = 0;
    if (ep.absmax) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < valid) top = max(top, mag_bits(o[i]));
    }
    return top;
}
template <class T, int ACT>
__device__ __forceinline__ uint32_t finish_gated8(const v4i &glo, const v4i &ghi, const v4i &ulo, const v4i &uhi,
                                                  const Epi &ep, int e2, const float (&bg)[8], const float (&bu)[8],
                                                  int64_t m, int n, int M, int H) {
    const int g[8] = {glo.x, glo.y, glo.z, glo.w, ghi.x, ghi.y, ghi.z, ghi.w};
    const int u[8] = {ulo.x, ulo.y, ulo.z, ulo.w, uhi.x, uhi.y, uhi.z, uhi.w};
    return finish_gated<T, ACT, 8>(g, u, ep, e2, bg, bu, m, n, M, H);
}
template <class T, int ACT>
__device__ __forceinline__ uint32_t finish_gated4(const v4i &sg, const v4i &su, const Epi &ep, int e2,
                                                  const float (&bg)[4], const float (&bu)[4], int64_t m, int n, int M,
                                                  int H) {
    const int g[4] = {sg.x, sg.y, sg.z, sg.w}, u[4] = {su.x, su.y, su.z, su.w};
    return finish_gated<T, ACT, 4>(g, u, ep, e2, bg, bu, m, n, M, H);
}

// Four sums of row m, columns n .. n + 3, through the epilogue (b: the
// columns' bias); returns the largest magnitude's bits of y (of the columns
// that exist).  LINEAR: no bias, activation, residual or z (the gradients'
// products).
template <class T, int ACT, bool LINEAR>
__device__ __forceinline__ uint32_t finish4(const v4i &s, const Epi &ep, int e2, const float (&b)[4], int64_t m, int n,
                                            int M, int N) {
    if (m >= M || n >= N) return 0u;
    const int valid = N - n;
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = __builtin_amdgcn_ldexpf(float(s[i]), e2);
    const int64_t at = m * N + n;
    T *y = static_cast<T *>(ep.y) + at;
    if (LINEAR) {
        store_vec<T, 4>(y, z, valid);
        return 0u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] += b[i];
    if (ep.z) store_vec<T, 4>(static_cast<T *>(ep.z) + at, z, valid);
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = act_value<ACT, kTermsValue<T>>(z[i]);
    if (ep.residual) {
        const auto r = load_raw<T, 4>(static_cast<const T *>(ep.residual) + at, valid);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += float(r[i]);
    }
    store_vec<T, 4>(y, o, valid);
    uint32_t top = 0;
    if (ep.absmax) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < valid) top = max(top, mag_bits(o[i]));
    }
    return top;
}

// Row m, columns n .. n + 7 of the sums through the epilogue; b: the columns'
// bias.
template <class T, int ACT, bool LINEAR>
__device__ __forceinline__ uint32_t finish8(const v4i &lo, const v4i &hi, const Epi &ep, int e2, const float (&b)[8],
                                            int64_t m, int n, int M, int N) {
    if (m >= M || n >= N) return 0u;
    const int valid = N - n;
    float z[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        z[i] = __builtin_amdgcn_ldexpf(float(lo[i]), e2);
        z[4 + i] = __builtin_amdgcn_ldexpf(float(hi[i]), e2);
    }
    const int64_t at = m * N + n;
    T *y = static_cast<T *>(ep.y) + at;
    if (LINEAR) {
        store_vec<T, 8>(y, z, valid);
        return 0u;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += b[i];
    if (ep.z) store_vec<T, 8>(static_cast<T *>(ep.z) + at, z, valid);
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = act_value<ACT, kTermsValue<T>>(z[i]);
    if (ep.residual) {
        const auto r = load_raw<T, 8>(static_cast<const T *>(ep.residual) + at, valid);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += float(r[i]);
    }
    store_vec<T, 8>(y, o, valid);
    uint32_t top = 0;
    if (ep.absmax) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) top = max(top, mag_bits(o[i]));
    }
    return top;
}

// The sums of one tile over k in [k_begin, k_end) (k_begin and, but for the
// last range, k_end multiples of BK).  lds: 2 stages of (BM + BN) * BK bytes.
template <int BM, int BN, int DEPTH, bool A_KM, bool B_KM, bool TINY, bool GATED = false>
__device__ __forceinline__ void tile_sums(const int8_t *__restrict__ A, int64_t lda, const int8_t *__restrict__ B,
                                          int64_t ldb, int M, int N, int m0, int n0, int k_begin, int k_end, int8_t *lds,
                                          int wm, int wn, int lane, v16i (&acc)[BM / 64][BN / 64]) {
    constexpr int FM = BM / 64, FN = BN / 64;  // 32 x 32 blocks of a wavefront
    constexpr int kStage = (BM + BN) * BK;
    static_assert(DEPTH % 2 == 0, "two LDS stages: DEPTH steps unrolled keep every index static");
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = v16i{};
    const int nk = (k_end - k_begin + BK - 1) / BK;
    if (nk <= 0) return;
    Stage<BM, A_KM, TINY> sa[DEPTH];
    Stage<BN, B_KM, TINY, GATED> sb[DEPTH];
    auto load = [&](int s, int kt) __attribute__((always_inline)) {
        sa[s].load(A, lda, M, k_end, m0, k_begin + kt * BK);
        sb[s].load(B, ldb, N, k_end, n0, k_begin + kt * BK);
    };
    auto store = [&](int s, int kt, int8_t *to) __attribute__((always_inline)) {
        sa[s].store(to, M, k_end, m0, k_begin + kt * BK);
        sb[s].store(to + BM * BK, N, k_end, n0, k_begin + kt * BK);
    };
    // (a load past the last step would repeat its pieces: skipped, for all lanes)
#pragma unroll
    for (int s = 0; s < DEPTH; ++s)
        if (s < nk) load(s, s);
    store(0, 0, lds);
    if (DEPTH < nk) load(0, DEPTH);
    __syncthreads();
    for (int k4 = 0; k4 < nk; k4 += DEPTH) {
#pragma unroll
        for (int s = 0; s < DEPTH; ++s) {
            const int kt = k4 + s;
            if (kt >= nk) break;
            const int8_t *As = lds + (s & 1) * kStage, *Bs = As + BM * BK;
#pragma unroll
            for (int sl = 0; sl < BK / 32; ++sl) {
                v4i a[FM], b[FN];
#pragma unroll
                for (int i = 0; i < FM; ++i) a[i] = read_frag<BM, A_KM>(As, wm + 32 * i, sl, lane);
#pragma unroll
                for (int j = 0; j < FN; ++j) b[j] = read_frag<BN, B_KM>(Bs, wn + 32 * j, sl, lane);
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[j], a[i], acc[i][j], 0, 0, 0);
            }
            if (kt + 1 < nk) store((s + 1) % DEPTH, kt + 1, lds + ((s + 1) & 1) * kStage);
            if (kt + 1 + DEPTH < nk) load((s + 1) % DEPTH, kt + 1 + DEPTH);
            __syncthreads();
        }
    }
}

// (A gated layer's product has N = H outputs, B its 2 H rows of weights, and n0
// of a tile counts rows of both halves: outputs n0 / 2 ...)
//
// A product C [M][N] over K with its epilogue, cut into tiles and, where
// there are few of them over a long reduction, into `split` ranges of K: each
// range leaves its int32 sums in part [split][M][N], and sum_kernel adds them
// (exactly, so in any order) and applies the epilogue.
struct Product {
    const int8_t *A, *B;
    int64_t lda, ldb;
    Epi ep;
    int M, N, K;
    int split;      // 1: the tiles apply the epilogue themselves
    int32_t *part;  // nullable when split is 1
    int blocks;     // workgroups: tiles * split
};

template <int BM, int BN>
constexpr int kTileLds = 2 * (BM + BN) * BK;

// Eight sums of row m at columns n .. of a range's [M][N] part.
__device__ __forceinline__ void store_part8(int32_t *row, const v4i &lo, const v4i &hi, int valid) {
    typedef v4i loose __attribute__((aligned(4)));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const v4i s = h ? hi : lo;
        if (4 * h + 4 <= valid) {
            *reinterpret_cast<loose *>(row + 4 * h) = s;
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (4 * h + e < valid) row[4 * h + e] = s[e];
        }
    }
}

// A gated layer's tile, its sums in LDS as run_tile lays them: BN / 2 outputs
// from n0 on, their gate sums in the first columns and the up sums in the others.
// Ranges leave theirs in part [split][M][2 H].
template <class T, int BM, int BN>
__device__ __forceinline__ void finish_gated_tile(const Product &p, const v4i *buf, int range, int m0, int n0) {
    constexpr int kPieces = BN / 4, kLanes = BN / 16, kRows = NT / kLanes;
    const int M = p.M, H = p.N;
    const int c = 2 * (int(threadIdx.x) % kLanes), n = n0 + 4 * c, r0 = int(threadIdx.x) / kLanes;
    const Epi &ep = p.ep;
    int32_t *part = p.part + int64_t(range) * M * 2 * H;
    const int e2 = *ep.ea + *ep.eb;
    float bg[8] = {}, bu[8] = {};
    if (p.split == 1 && n < H) load_bias2(ep, n, H, bg, bu);
    uint32_t top = 0;
    with_act(ep.act, [&](auto ac) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < BM / kRows; ++k) {
            const int r = kRows * k + r0;
            const int64_t m = int64_t(m0) + r;
            const auto at = [&](int i) __attribute__((always_inline)) { return buf[r * kPieces + ((c + i) ^ (r & 15))]; };
            const v4i glo = at(0), ghi = at(1), ulo = at(kPieces / 2), uhi = at(kPieces / 2 + 1);
            if (p.split > 1) {
                if (m < M && n < H) {
                    store_part8(part + 2 * m * H + n, glo, ghi, H - n);
                    store_part8(part + 2 * m * H + H + n, ulo, uhi, H - n);
                }
            } else {
                top = max(top, finish_gated8<T, decltype(ac)::value>(glo, ghi, ulo, uhi, ep, e2, bg, bu, m, n, M, H));
            }
        }
    });
    if (ep.absmax && p.split == 1) {
        top = wave_max_u32(top);
        if ((threadIdx.x & 63) == 0) publish_max_u32(ep.absmax, top);
    }
}

// Workgroup `id` of a product: the tile id % tiles over range id / tiles.
template <class T, int BM, int BN, int DEPTH, bool A_KM, bool B_KM, bool LINEAR, bool TINY, bool GATED = false>
__device__ __forceinline__ void run_tile(const Product &p, int id, int8_t *lds) {
    constexpr int FM = BM / 64, FN = BN / 64;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int wm = (wave >> 1) * (BM / 2), wn = (wave & 1) * (BN / 2);
    const int M = p.M, N = p.N;
    // the range of K (scalar divisions cost tens of instructions each: only
    // where there are ranges)
    int range = 0, tile = id, k_begin = 0, k_end = p.K;
    if (p.split > 1) {
        const uint32_t tiles = uint32_t(p.blocks) / uint32_t(p.split), steps = uint32_t(p.K + BK - 1) / BK;
        range = int(uint32_t(id) / tiles);
        tile = id - range * int(tiles);
        k_begin = int(steps * uint32_t(range) / uint32_t(p.split)) * BK;  // steps <= 1024, split <= 32
        k_end = min(p.K, int(steps * uint32_t(range + 1) / uint32_t(p.split)) * BK);
    }
    int tm, tn;
    constexpr int kCols = GATED ? BN / 2 : BN;  // outputs of a tile
    gemm::tile_coords(tile, (M + BM - 1) / BM, (N + kCols - 1) / kCols, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    v16i acc[FM][FN];
    tile_sums<BM, BN, DEPTH, A_KM, B_KM, TINY, GATED>(p.A, p.lda, p.B, p.ldb, M, N, m0, n0, k_begin, k_end, lds, wm, wn, lane,
                                               acc);
    // The tile through LDS (lane: row lane % 32, columns 8 q + 4 (lane / 32)
    // .. + 3 of each 32 x 32 block; 16-byte piece c of row r at position c ^ (r
    // & 15), free of bank conflicts), so that a thread finishes eight columns
    // and a row's run of 128 bytes or more leaves together.
    static_assert(BM * BN * 4 <= kTileLds<BM, BN>, "the sums fit where the stages were");
    constexpr int kPieces = BN / 4;  // of a row
    v4i *buf = reinterpret_cast<v4i *>(lds);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = wm + 32 * i + (lane & 31), c = (wn + 32 * j) / 4 + 2 * q + (lane >> 5);
                buf[r * kPieces + (c ^ (r & 15))] =
                    v4i{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            }
    __syncthreads();
    if constexpr (GATED) {
        finish_gated_tile<T, BM, BN>(p, buf, range, m0, n0 / 2);
        return;
    }
    const int c = 2 * (int(threadIdx.x) % (BN / 8)), n = n0 + 4 * c;  // the thread's eight columns
    constexpr int kRows = NT / (BN / 8);                              // rows finished at once
    if (p.split > 1) {
        typedef v4i loose __attribute__((aligned(4)));
        int32_t *part = p.part + int64_t(range) * M * N;
#pragma unroll
        for (int k = 0; k < BM / kRows; ++k) {
            const int r = kRows * k + int(threadIdx.x) / (BN / 8);
            const int64_t m = int64_t(m0) + r;
            if (m >= M) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4i s = buf[r * kPieces + ((c + h) ^ (r & 15))];
                const int nh = n + 4 * h;
                if (nh + 4 <= N) {
                    *reinterpret_cast<loose *>(part + m * N + nh) = s;
                } else {
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        if (nh + e < N) part[m * N + nh + e] = s[e];
                }
            }
        }
        return;
    }
    const Epi &ep = p.ep;
    const int e2 = *ep.ea + *ep.eb;
    float bias[8] = {};
    if (!LINEAR) load_bias(ep, n, N, bias);
    uint32_t top = 0;
    with_act(LINEAR ? int(IONN_ACT_NONE) : ep.act, [&](auto ac) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < BM / kRows; ++k) {
            const int r = kRows * k + int(threadIdx.x) / (BN / 8);
            const v4i lo = buf[r * kPieces + (c ^ (r & 15))], hi = buf[r * kPieces + ((c + 1) ^ (r & 15))];
            top = max(top, finish8<T, decltype(ac)::value, LINEAR>(lo, hi, ep, e2, bias, int64_t(m0) + r, n, M, N));
        }
    });
    if (!LINEAR && ep.absmax) {
        top = wave_max_u32(top);
        if (lane == 0) publish_max_u32(ep.absmax, top);
    }
}

template <class T, int BM, int BN, int DEPTH, bool A_KM, bool B_KM, bool LINEAR, bool TINY, bool GATED = false>
__global__ __launch_bounds__(NT) void tile_kernel(Product p) {
    __shared__ __attribute__((aligned(256))) int8_t lds[kTileLds<BM, BN>];
    run_tile<T, BM, BN, DEPTH, A_KM, B_KM, LINEAR, TINY, GATED>(p, int(blockIdx.x), lds);
}

// The two products of a backward pass in one launch: dX's workgroups, then
// G's (a product that is not asked for has none).
template <class T, int BM, int BN, int DEPTH>
__global__ __launch_bounds__(NT) void tile_pair_kernel(Product d, Product g) {
    __shared__ __attribute__((aligned(256))) int8_t lds[kTileLds<BM, BN>];
    if (int(blockIdx.x) < d.blocks)
        run_tile<T, BM, BN, DEPTH, true, false, true, false>(d, int(blockIdx.x), lds);
    else
        run_tile<T, BM, BN, DEPTH, false, false, true, false>(g, int(blockIdx.x) - d.blocks, lds);
}

// The sums of the ranges through the epilogue, four columns of a row per
// thread; element `id` of the product's M * ceil(N / 4) (below 2^31: only
// products of few tiles are cut into ranges).
template <class T, bool LINEAR>
__device__ __forceinline__ void sum_ranges(const Product &p, uint32_t id) {
    typedef v4i loose __attribute__((aligned(4)));
    const uint32_t n4 = uint32_t(p.N + 3) / 4;
    const uint32_t row = id / n4;
    const int n = 4 * int(id - row * n4);
    const int64_t m = row;
    uint32_t top = 0;
    if (m < p.M) {
        const int32_t *at = p.part + m * p.N + n;
        const int64_t step = int64_t(p.M) * p.N;
        v4i s = {0, 0, 0, 0};
        if (n + 4 <= p.N) {
#pragma unroll 4
            for (int r = 0; r < p.split; ++r) s += *reinterpret_cast<const loose *>(at + r * step);
        } else {
            for (int r = 0; r < p.split; ++r)
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (n + e < p.N) s[e] += at[r * step + e];
        }
        const int e2 = *p.ep.ea + *p.ep.eb;
        float bias[4] = {};
        if (!LINEAR) load_bias(p.ep, n, p.N, bias);
        with_act(LINEAR ? int(IONN_ACT_NONE) : p.ep.act, [&](auto ac) __attribute__((always_inline)) {
            top = finish4<T, decltype(ac)::value, LINEAR>(s, p.ep, e2, bias, m, n, p.M, p.N);
        });
    }
    if (!LINEAR && p.ep.absmax) {
        top = wave_max_u32(top);
        if ((threadIdx.x & 63) == 0) publish_max_u32(p.ep.absmax, top);
    }
}

// The same of a gated layer's halves, from part [split][M][2 H].
template <class T>
__global__ __launch_bounds__(NT) void sum_gated_kernel(Product p) {
    const uint32_t id = blockIdx.x * NT + threadIdx.x, n4 = uint32_t(p.N + 3) / 4, row = id / n4;
    const int n = 4 * int(id - row * n4), H = p.N, valid = H - n;
    const int64_t m = row, step = int64_t(p.M) * 2 * H;
    uint32_t top = 0;
    if (m < p.M) {
        typedef v4i loose __attribute__((aligned(4)));
        v4i s[2] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int32_t *at = p.part + 2 * m * H + h * H + n;
            for (int r = 0; r < p.split; ++r, at += step) {
                if (valid >= 4) {
                    s[h] += *reinterpret_cast<const loose *>(at);
                } else {
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        if (e < valid) s[h][e] += at[e];
                }
            }
        }
        const int e2 = *p.ep.ea + *p.ep.eb;
        float bg[4], bu[4];
        load_bias2(p.ep, n, H, bg, bu);
        with_act(p.ep.act, [&](auto ac) __attribute__((always_inline)) {
            top = finish_gated4<T, decltype(ac)::value>(s[0], s[1], p.ep, e2, bg, bu, m, n, p.M, H);
        });
    }
    if (p.ep.absmax) {
        top = wave_max_u32(top);
        if ((threadIdx.x & 63) == 0) publish_max_u32(p.ep.absmax, top);
    }
}

template <class T, bool LINEAR>
__global__ __launch_bounds__(NT) void sum_kernel(Product p) {
    sum_ranges<T, LINEAR>(p, blockIdx.x * NT + threadIdx.x);
}

// The same for the two products of a backward pass (workgroups of the first,
// d_groups of them, then the second's).
template <class T>
__global__ __launch_bounds__(NT) void sum_pair_kernel(Product d, Product g, int d_groups) {
    if (int(blockIdx.x) < d_groups) sum_ranges<T, true>(d, blockIdx.x * NT + threadIdx.x);
    else sum_ranges<T, true>(g, (blockIdx.x - uint32_t(d_groups)) * NT + threadIdx.x);
}

}  // namespace dfp8
}  // namespace ionn
