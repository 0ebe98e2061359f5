// The large-product path of the DFP-8 Linear layer: 256 x 256 output tiles,
// 128-deep K steps, loads straight into LDS, on the operand layouts, fragment
// reads and issue order of gemm256.h, with a floating epilogue and with edges:
// any sizes whose row pitches are multiples of 16, so that 16-byte pieces stay
// aligned.
//
// Bound by the matrix cores at the clock that their power leaves: 8192 x 4096
// x 4096 takes 128 us as dX (2140 TOP/s) and 116 us as G (2370 TOP/s), where
// the library's int8 product reaches 2030 TOP/s on 8192^3; forward with gelu and
// z 150 us, the epilogue's arithmetic (24 instructions per output, one
// wavefront per SIMD) not overlapping the products.
//
// Edges cost no branch.  Rows past a K-major operand's end and k past an
// M-major one's lie past its buffer resource and come back as zeros; what a
// row's or column's end lets in of the next row feeds outputs that are not
// stored.  Only where both operands are K-major does k past the end meet the
// next row on both sides: there A's pieces past K are sent out of range.  An
// address is a per-lane offset alone (no scalar offset): the hardware's range
// check subtracts a scalar offset from the resource's size, which wraps when
// a whole instruction lies past the end.
#pragma once

#include "dfp8_tile.h"

namespace ionn {
namespace dfp8 {

constexpr uint32_t kOut = 0x80000000u;  // past every resource, also with an offset below 2^31 added

// The per-lane offsets of one operand (TileSrc holds the resource, the pitch
// and the wavefront's and lanes' positions).
template <bool KMAJOR>
struct EdgeSrc : g256::TileSrc<KMAJOR> {
    int col[2];  // K-major: the piece's first k within a step
    __device__ __forceinline__ void init_edge(const int8_t *b, int ld, uint32_t bytes, int r0, int wave, int lane) {
        this->init(b, ld, bytes, r0, wave, lane);
#pragma unroll
        for (int p = 0; p < 2; ++p) col[p] = 16 * ((lane & 7) ^ g256::fK(8 * p + (lane >> 3)));
    }
    // lane offsets of a step whose first k is K - left (MASK: pieces past K out of range)
    template <bool MASK>
    __device__ __forceinline__ void offsets(int left, uint32_t (&v)[2]) const {
#pragma unroll
        for (int p = 0; p < 2; ++p) v[p] = !MASK || col[p] < left ? this->lane_off[p] : kOut;
    }
    __device__ __forceinline__ void one(const uint32_t (&v)[2], int k0, int8_t *dst, int wave, int qq) const {
        g256::dma16(this->rsrc, v[qq & 1] + this->soff_of(k0, qq), 0u, this->lds_of(dst, wave, qq));
    }
    __device__ __forceinline__ void two(const uint32_t (&v)[2], int k0, int8_t *dst, int wave, int qq) const {
        g256::dma16x2(this->rsrc, v[0] + this->soff_of(k0, qq), 0u, v[1] + (this->soff_of(k0, qq + 1) - 1024u), 0u,
                      this->lds_of(dst, wave, qq));
    }
};

// The epilogue of a wavefront's 128 x 128 sums, 64 columns at a time through
// 32 KiB of LDS: the accumulators are written as they lie (lane: row lane %
// 32, columns 8 q + 4 (lane / 32) .. + 3 of each 32 x 32 block; 16-byte piece
// c of row r at position c ^ (r & 15), free of bank conflicts both ways) and
// read back eight columns a lane, so that a loop of a few hundred
// instructions writes whole 128-byte lines of a 16-bit output.  Unrolled over
// the registers the same epilogue was 60 KB of straight code per activation,
// whose fetching took longer than its work (8192 x 4096 x 4096 with gelu and z:
// 208 us against 171 with the same arithmetic).
template <class T, int ACT, bool LINEAR>
__device__ __forceinline__ uint32_t finish_wave(const v16i (&acc)[4][4], int8_t *lds, const Epi &ep, int e2, int64_t m0,
                                                int n0, int M, int N, int lane) {
    uint32_t top = 0;
    v4i *buf = reinterpret_cast<v4i *>(lds);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const v16i &a = acc[i][2 * h + j];
                    const int r = 32 * i + (lane & 31), c = 8 * j + 2 * q + (lane >> 5);
                    buf[16 * r + (c ^ (r & 15))] = v4i{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
                }
        const int c = 2 * (lane & 7), n = n0 + 64 * h + 8 * (lane & 7);
        float b[8] = {};
        if (!LINEAR) load_bias(ep, n, N, b);
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the wavefront's own writes
        __builtin_amdgcn_wave_barrier();
#pragma unroll 2
        for (int k = 0; k < 16; ++k) {
            const int r = 8 * k + (lane >> 3);
            const v4i lo = buf[16 * r + (c ^ (r & 15))], hi = buf[16 * r + ((c + 1) ^ (r & 15))];
            top = max(top, finish8<T, ACT, LINEAR>(lo, hi, ep, e2, b, m0 + r, n, M, N));
        }
        __builtin_amdgcn_wave_barrier();
    }
    return top;
}

template <class T, bool A_KM, bool B_KM, bool LINEAR>
__global__ __launch_bounds__(g256::NT, 1) void tile256_kernel(const int8_t *__restrict__ A, int64_t lda,
                                                              const int8_t *__restrict__ B, int64_t ldb,
                                                              uint32_t a_bytes, uint32_t b_bytes, Epi ep, int M, int N,
                                                              int K) {
    using namespace g256;
    __shared__ __attribute__((aligned(1024))) int8_t sA0[TILE_BYTES];
    __shared__ __attribute__((aligned(1024))) int8_t sB0[TILE_BYTES];
    __shared__ __attribute__((aligned(1024))) int8_t sA1[TILE_BYTES];
    __shared__ __attribute__((aligned(1024))) int8_t sB1[TILE_BYTES];
    constexpr bool MASK = A_KM && B_KM;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    int tm, tn;
    gemm::tile_coords(blockIdx.x, (M + BM - 1) / BM, (N + BN - 1) / BN, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;

    EdgeSrc<A_KM> ta;
    EdgeSrc<B_KM> tb;
    ta.init_edge(A, int(lda), a_bytes, m0, wave, lane);
    tb.init_edge(B, int(ldb), b_bytes, n0, wave, lane);
    FragSrc<A_KM> fa;
    FragSrc<B_KM> fb;
    fa.init(wm * 128, lane);
    fb.init(wn * 128, lane);
    const int e2 = *ep.ea + *ep.eb;

    v16i acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v16i{};
    Frags<A_KM, B_KM> F[2];
    const int nk = 2 * ((K + 2 * g256::BK - 1) / (2 * g256::BK));  // the two stages take turns: an even count

    // va: A's lane offsets of the step being loaded
    uint32_t va[2];
    const uint32_t(&vb)[2] = tb.lane_off;
    auto dma1 = [&](int q, int k0, int8_t *Ad, int8_t *Bd) __attribute__((always_inline)) {
        if (q < 8) ta.one(va, k0, Ad, wave, q);
        else tb.one(vb, k0, Bd, wave, q - 8);
    };
    auto dma2 = [&](int q, int k0, int8_t *Ad, int8_t *Bd) __attribute__((always_inline)) {
        if (q < 8) ta.two(va, k0, Ad, wave, q);
        else tb.two(vb, k0, Bd, wave, q - 8);
    };
    ta.template offsets<MASK>(K, va);
#pragma unroll
    for (int q = 0; q < 16; q += 2) dma2(q, 0, sA0, sB0);
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    ta.template offsets<MASK>(K - g256::BK, va);
    dma2(0, g256::BK, sA1, sB1);
    dma2(2, g256::BK, sA1, sB1);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
#pragma unroll
    for (int r = 0; r < 8; ++r) F[0].read(RO[r], sA0, sB0, fa, fb, 0);

    // One K step, in the issue order of gemm256_kernel: one memory
    // instruction between consecutive MFMAs, the step's stage read while the
    // other stage receives the next step, whose first four loads went out at
    // the end of the step before.
    auto step = [&](const int8_t *Ac, const int8_t *Bc, const int8_t *An, const int8_t *Bn, int8_t *Adst, int8_t *Bdst,
                    int kt) __attribute__((always_inline)) {
        int8_t *Anw = const_cast<int8_t *>(An), *Bnw = const_cast<int8_t *>(Bn);
        const bool more1 = kt + 1 < nk, more2 = kt + 2 < nk;
#pragma unroll
        for (int sl = 0; sl < 3; ++sl) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = 4 * sl + g;
                mfma_gt(F[sl & 1], g, 0, acc);
                IONN_SCHED_FENCE();
                F[(sl + 1) & 1].read(RO[2 * g], Ac, Bc, fa, fb, sl + 1);
                IONN_SCHED_FENCE();
                mfma_gt(F[sl & 1], g, 1, acc);
                IONN_SCHED_FENCE();
                if (c < 8 && more1) {
                    if (c < 4) dma2(4 + 2 * c, (kt + 1) * g256::BK, Anw, Bnw);
                    else dma1(12 + (c - 4), (kt + 1) * g256::BK, Anw, Bnw);
                }
                IONN_SCHED_FENCE();
                mfma_gt(F[sl & 1], g, 2, acc);
                IONN_SCHED_FENCE();
                F[(sl + 1) & 1].read(RO[2 * g + 1], Ac, Bc, fa, fb, sl + 1);
                IONN_SCHED_FENCE();
                mfma_gt(F[sl & 1], g, 3, acc);
                IONN_SCHED_FENCE();
            }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) mfma_gt(F[1], t >> 2, t & 3, acc);
        IONN_SCHED_FENCE();
        ta.template offsets<MASK>(K - (kt + 2) * g256::BK, va);
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        IONN_SCHED_FENCE();
#pragma unroll
        for (int g = 2; g < 4; ++g) {
            if (more2) dma2(2 * (g - 2), (kt + 2) * g256::BK, Adst, Bdst);
            IONN_SCHED_FENCE();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                mfma_gt(F[1], g, t, acc);
                IONN_SCHED_FENCE();
                F[0].read(RO[4 * (g - 2) + t], An, Bn, fa, fb, 0);
                IONN_SCHED_FENCE();
            }
        }
    };
    for (int kt = 0; kt < nk; kt += 2) {
        step(sA0, sB0, sA1, sB1, sA0, sB0, kt);
        step(sA1, sB1, sA0, sB0, sA1, sB1, kt + 1);
    }

    // every wavefront is done with the stages: 32 KiB of them for each
    __builtin_amdgcn_s_waitcnt(0xc07f);
    __builtin_amdgcn_s_barrier();
    int8_t *mine = wave == 0 ? sA0 : wave == 1 ? sB0 : wave == 2 ? sA1 : sB1;
    uint32_t top = 0;
    with_act(LINEAR ? int(IONN_ACT_NONE) : ep.act, [&](auto ac) __attribute__((always_inline)) {
        top = finish_wave<T, decltype(ac)::value, LINEAR>(acc, mine, ep, e2, int64_t(m0) + wm * 128, n0 + wn * 128, M, N,
                                                          lane);
    });
    if (!LINEAR && ep.absmax) {
        top = wave_max_u32(top);
        if (lane == 0) publish_max_u32(ep.absmax, top);
    }
}

// Whether tile256_kernel takes the product: 16-byte pieces that stay aligned,
// offsets of a tensor's rows that stay below 2^31 with a step added, and of a
// ragged tile's below 2^32.
template <bool A_KM, bool B_KM>
inline bool tile256_fits(const int8_t *A, int64_t lda, const int8_t *B, int64_t ldb, int64_t M, int64_t N, int64_t K) {
    const int64_t ab = (A_KM ? M : K) * lda, bb = (B_KM ? N : K) * ldb, lim = (int64_t(1) << 31) - 1024;
    return K >= 1 && aligned(A, 16) && aligned(B, 16) && lda % 16 == 0 && ldb % 16 == 0 && ab < lim && bb < lim &&
           512 * lda < lim && 512 * ldb < lim && lda >= 256 && ldb >= 256;
}

}  // namespace dfp8
}  // namespace ionn
