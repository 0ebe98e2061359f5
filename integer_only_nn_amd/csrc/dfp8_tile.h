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
// steps, double-buffered in LDS; the next step's 16-byte pieces are loaded
// into registers while the current step is contracted.  Pieces are loaded at
// whatever byte they start on, and a piece that a row's (or the tensor's) end
// cuts is loaded so that it ends there and shifted down, so odd sizes cost a
// shift in the last piece and no byte-wise path.
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

template <int R>
__device__ __forceinline__ int fT(int k) {
    return R == 128 ? 2 * ((k >> 1) & 3) : 2 * ((k >> 2) & 1);
}

// One operand's tile of R rows: pieces to registers, then to LDS.
template <int R, bool KMAJOR>
struct Stage {
    static constexpr int kPer = R * BK / 16 / NT;
    static_assert(R * BK / 16 % NT == 0, "whole pieces per thread");
    v4i reg[kPer];
    __device__ __forceinline__ void load(const int8_t *base, int64_t ld, int rows, int kdim, int r0, int k0) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int id = j * NT + int(threadIdx.x);
            if (KMAJOR) {
                const int r = r0 + id / (BK / 16), k = k0 + 16 * (id % (BK / 16));
                reg[j] = load_piece(base, r * ld + k, r < rows ? kdim - k : 0);
            } else {
                const int k = k0 + id / (R / 16), r = r0 + 16 * (id % (R / 16));
                reg[j] = load_piece(base, k * ld + r, k < kdim ? rows - r : 0);
            }
        }
    }
    __device__ __forceinline__ void store(int8_t *lds) const {
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

// Four sums of row m, columns n .. n + 3, through the epilogue; returns the
// largest magnitude's bits of y (of the columns that exist).  LINEAR: no
// bias, activation, residual or z (the gradients' products).
template <class T, int ACT, bool LINEAR>
__device__ __forceinline__ uint32_t finish4(const v4i &s, const Epi &ep, int e2, int64_t m, int n, int M, int N) {
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
    if (ep.bias) {
        const auto b = load_raw<float, 4>(ep.bias + n, valid);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] += b[i];
    }
    if (ep.z) store_vec<T, 4>(static_cast<T *>(ep.z) + at, z, valid);
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = act_value<ACT>(z[i]);
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

template <class T, int BM, int BN, bool A_KM, bool B_KM, bool LINEAR>
__global__ __launch_bounds__(NT) void tile_kernel(const int8_t *__restrict__ A, int64_t lda,
                                                  const int8_t *__restrict__ B, int64_t ldb, Epi ep, int M, int N,
                                                  int K) {
    constexpr int FM = BM / 64, FN = BN / 64;  // 32 x 32 blocks of a wavefront
    __shared__ __attribute__((aligned(256))) int8_t lds[2][(BM + BN) * BK];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int wm = (wave >> 1) * (BM / 2), wn = (wave & 1) * (BN / 2);
    int tm, tn;
    gemm::tile_coords(blockIdx.x, (M + BM - 1) / BM, (N + BN - 1) / BN, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    v16i acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = v16i{};
    Stage<BM, A_KM> sa;
    Stage<BN, B_KM> sb;
    const int nk = (K + BK - 1) / BK;
    if (nk > 0) {
        sa.load(A, lda, M, K, m0, 0);
        sb.load(B, ldb, N, K, n0, 0);
        sa.store(lds[0]);
        sb.store(lds[0] + BM * BK);
    }
    __syncthreads();
    for (int kt = 0; kt < nk; ++kt) {
        const int8_t *As = lds[kt & 1], *Bs = As + BM * BK;
        const bool more = kt + 1 < nk;
        if (more) {
            sa.load(A, lda, M, K, m0, (kt + 1) * BK);
            sb.load(B, ldb, N, K, n0, (kt + 1) * BK);
        }
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
        if (more) {
            int8_t *nx = lds[(kt + 1) & 1];
            sa.store(nx);
            sb.store(nx + BM * BK);
        }
        __syncthreads();
    }
    // lane: row lane % 32, columns 8 q + 4 (lane / 32) .. + 3 of each block
    const int e2 = *ep.ea + *ep.eb;
    uint32_t top = 0;
    with_act(LINEAR ? int(IONN_ACT_NONE) : ep.act, [&](auto ac) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const v4i s = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                    top = max(top, finish4<T, decltype(ac)::value, LINEAR>(
                                       s, ep, e2, int64_t(m0) + wm + 32 * i + (lane & 31),
                                       n0 + wn + 32 * j + 8 * q + 4 * (lane >> 5), M, N));
                }
    });
    if (!LINEAR && ep.absmax) {
        top = wave_max_u32(top);
        if (lane == 0) publish_max_u32(ep.absmax, top);
    }
}

}  // namespace dfp8
}  // namespace ionn
